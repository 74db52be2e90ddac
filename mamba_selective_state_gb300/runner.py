"""Device buffers for one SSD problem and the calls that run it through the
C ABI.  Allocation and argument marshalling only; the layer runs in libssd.
"""
from __future__ import annotations

import contextlib
import functools

import torch

from . import _lib
from .inputs import NormInputs, SSDInputs


class SSDDevice:
    """Inputs copied to ``device``, outputs, gradients and workspace allocated.

    ``dfinal``/``want_dinit`` select the optional backward arguments; by
    default they follow the inputs (dfinal_states present -> used; initial
    states present -> dinitial_states wanted)."""

    def __init__(self, inp: SSDInputs, device="cuda", backward=True, dfinal=None,
                 want_dinit=None, extra_flags=0):
        self.inp = inp
        self.device = torch.device(device)
        dev = self.device
        to = lambda t: None if t is None else t.to(dev).contiguous()  # noqa: E731
        self.x, self.dt, self.B, self.C = to(inp.x), to(inp.dt), to(inp.B), to(inp.C)
        self.dt_bias, self.A, self.D = to(inp.dt_bias), to(inp.A), to(inp.D)
        self.init = to(inp.initial_states)
        self.seq_idx = to(inp.seq_idx)
        use_dfinal = (inp.dfinal_states is not None) if dfinal is None else dfinal
        self.dfinal = to(inp.dfinal_states) if use_dfinal else None
        self.want_dinit = (inp.initial_states is not None) if want_dinit is None else want_dinit
        self.dy = to(inp.dy) if backward else None
        dt_t = inp.torch_dtype
        b, L, H, P, N, G = inp.batch, inp.seqlen, inp.nheads, inp.headdim, inp.dstate, inp.ngroups
        flags = extra_flags
        if self.init is not None:
            flags |= _lib.SSD_HAS_INIT
        if self.seq_idx is not None:
            flags |= _lib.SSD_HAS_SEQ_IDX
        self.fwd_prob = _lib.make_problem(b, L, H, P, N, G, inp.chunk, dt_t, flags)
        bflags = flags
        if self.dfinal is not None:
            bflags |= _lib.SSD_HAS_DFINAL
        if self.want_dinit:
            bflags |= _lib.SSD_WANT_DINIT
        self.bwd_prob = _lib.make_problem(b, L, H, P, N, G, inp.chunk, dt_t, bflags)
        self.y = torch.empty((b, L, H, P), dtype=dt_t, device=dev)
        self.final = torch.empty((b, H, P, N), dtype=torch.float32, device=dev)
        ws = _lib.ssd_bwd_workspace_bytes(self.bwd_prob) if backward else \
            _lib.ssd_fwd_workspace_bytes(self.fwd_prob)
        if ws == 0:
            raise _lib.SSDError(_lib.SSD_ERR_INVALID_ARGUMENT, "workspace size")
        self.workspace = torch.empty(ws, dtype=torch.uint8, device=dev)
        if backward:
            self.dx = torch.empty_like(self.x)
            self.ddt = torch.empty_like(self.dt)
            self.dB = torch.empty_like(self.B)
            self.dC = torch.empty_like(self.C)
            self.ddt_bias = torch.empty(H, dtype=torch.float32, device=dev)
            self.dA = torch.empty(H, dtype=torch.float32, device=dev)
            self.dD = torch.empty(H, dtype=torch.float32, device=dev)
            self.dinit = (torch.empty((b, H, P, N), dtype=torch.float32, device=dev)
                          if self.want_dinit else None)

    def fwd(self, stream=None, check=True):
        return _lib.ssd_fwd(self.fwd_prob, self.x, self.dt, self.dt_bias, self.A, self.B, self.C,
                            self.D, self.init, self.seq_idx, self.y, self.final, self.workspace,
                            stream=stream, check=check)

    def bwd(self, stream=None, check=True):
        return _lib.ssd_bwd(self.bwd_prob, self.x, self.dt, self.dt_bias, self.A, self.B, self.C,
                            self.D, self.init, self.seq_idx, self.dy, self.dfinal, self.dx,
                            self.ddt, self.ddt_bias, self.dA, self.dB, self.dC, self.dD,
                            self.dinit, self.workspace, stream=stream, check=check)

    def device_status(self, stream=None):
        return _lib.ssd_read_device_status(self.workspace, stream)

    def results(self) -> dict:
        """Outputs and gradients as CPU float64 tensors."""
        out = dict(y=self.y, final_states=self.final)
        if self.dy is not None:
            out.update(dx=self.dx, ddt=self.ddt, dB=self.dB, dC=self.dC, ddt_bias=self.ddt_bias,
                       dA=self.dA, dD=self.dD)
            if self.dinit is not None:
                out["dinitial_states"] = self.dinit
        return {k: v.detach().to("cpu", torch.float64) for k, v in out.items()}


class NormDevice:
    """Device buffers of one gated-RMSNorm problem (inputs, out, rstd, the
    gradients and the backward workspace) and its calls through the C ABI."""

    def __init__(self, inp: NormInputs, device="cuda"):
        self.inp = inp
        dev = torch.device(device)
        to = lambda t: None if t is None else t.to(dev).contiguous()  # noqa: E731
        self.y, self.z, self.weight, self.dout = to(inp.y), to(inp.z), to(inp.weight), to(inp.dout)
        self.prob = _lib.make_norm_problem(inp.rows, inp.dim, inp.group_size, inp.eps,
                                           inp.torch_dtype, gate=inp.z is not None)
        self.out = torch.empty_like(self.y)
        self.rstd = torch.empty((inp.rows, inp.dim // inp.group_size), dtype=torch.float32,
                                device=dev)
        self.dy = torch.empty_like(self.y)
        self.dz = None if self.z is None else torch.empty_like(self.z)
        self.dweight = torch.empty(inp.dim, dtype=torch.float32, device=dev)
        ws = _lib.ssd_gated_rmsnorm_bwd_workspace_bytes(self.prob)
        if ws == 0:
            raise _lib.SSDError(_lib.SSD_ERR_INVALID_ARGUMENT, "norm workspace size")
        self.workspace = torch.empty(ws, dtype=torch.uint8, device=dev)

    def fwd(self, stream=None, check=True):
        return _lib.ssd_gated_rmsnorm_fwd(self.prob, self.y, self.z, self.weight, self.out,
                                          self.rstd, stream=stream, check=check)

    def bwd(self, stream=None, check=True):
        return _lib.ssd_gated_rmsnorm_bwd(self.prob, self.y, self.z, self.weight, self.dout,
                                          self.dy, self.dz, self.dweight, self.workspace,
                                          stream=stream, check=check)

    def results(self) -> dict:
        out = dict(out=self.out, rstd=self.rstd, dy=self.dy, dweight=self.dweight)
        if self.dz is not None:
            out["dz"] = self.dz
        return {k: v.detach().to("cpu", torch.float64) for k, v in out.items()}


def _token_stride(shape, strides, inner, what):
    """Elements between the tokens of a (b, L, heads, d) tensor whose last two
    axes are dense and whose rows are L tokens long (a column block of a
    wider projection is one)."""
    b, L, heads, d = shape
    stride = strides[1] if L > 1 else strides[0] if b > 1 else inner
    if ((d > 1 and strides[3] != 1) or (heads > 1 and strides[2] != d)
            or (b > 1 and strides[0] != L * stride) or stride < inner):
        raise ValueError(f"{what}: its heads must be dense and its tokens evenly spaced")
    return stride


def _dense(t, shape, dtype, what, device=None):
    if t is not None and (t.shape != shape or t.dtype is not dtype or not t.is_contiguous()
                          or (device is not None and t.device != device)):
        raise ValueError(f"{what}: expected a dense {tuple(shape)} {dtype} tensor on {device}")


def _on_gpu(device, what):
    """The library gets bare pointers and launches on the current device: a
    tensor anywhere else would be read there at an address that is not its own."""
    if device.type != "cuda" or device.index != torch.cuda.current_device():
        raise ValueError(f"{what}: expected tensors on the current CUDA device, not on {device}")


def _allocating_on(stream):
    """Memory of a call's own outputs comes from the stream that fills them:
    the allocator hands out a block of another stream's as soon as that stream's
    later work may have it, which says nothing about this one's."""
    if stream is None:
        return contextlib.nullcontext()
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


_FLOATS = (torch.float32, torch.bfloat16)


# the problem structs of repeated shapes (the library only reads them)
_verify_problem = functools.lru_cache(maxsize=256)(_lib.make_verify_problem)
_cache_problem = functools.lru_cache(maxsize=256)(_lib.make_cache_problem)


@functools.lru_cache(maxsize=256)
def _delta_layout(meta):
    """(b, L, H, P, N, G) and the token strides of q, k, v from the tensors'
    shapes, strides, types and devices; raises where they do not fit."""
    (q, k, v, g, beta) = meta
    if len(v[0]) != 4 or len(q[0]) != 4 or v[2] not in _FLOATS:
        raise ValueError("v must be (b, L, H, P) and q (b, L, G, N), both fp32 or bf16")
    b, L, H, P = v[0]
    G, N = q[0][2:]
    for t, what in ((q, "q"), (k, "k")):
        if tuple(t[0]) != (b, L, G, N) or t[2:] != v[2:]:
            raise ValueError(f"{what}: expected a {(b, L, G, N)} {v[2]} tensor on {v[3]}")
    for t, what in ((g, "g"), (beta, "beta")):
        dense = (L * H, H, 1)
        if tuple(t[0]) != (b, L, H) or t[2:] != v[2:] or any(
                n > 1 and s != d for n, s, d in zip(t[0], t[1], dense)):
            raise ValueError(f"{what}: expected a dense {(b, L, H)} {v[2]} tensor on {v[3]}")
    strides = (_token_stride(q[0], q[1], G * N, "q"), _token_stride(k[0], k[1], G * N, "k"),
               _token_stride(v[0], v[1], H * P, "v"))
    return (b, L, H, P, N, G), strides


def _delta_shape(q, k, v, g, beta):
    return _delta_layout(tuple((t.shape, t.stride(), t.dtype, t.device)
                               for t in (q, k, v, g, beta)))


@functools.lru_cache(maxsize=256)
def _step_problem(shape, scale, dtype, strides):
    b, T, H, P, N, G = shape
    return _lib.make_delta_problem(b, T, H, P, N, G, scale, dtype, q_stride=strides[0],
                                   k_stride=strides[1], v_stride=strides[2])


class DeltaDevice:
    """One gated-delta-rule problem: the caller's device tensors, the outputs,
    the gradients (when ``dy`` is given), the workspace, and the calls through
    the C ABI.  q, k (b, L, G, N) and v (b, L, H, P) may be column blocks of
    one projection's output; g (log decay), beta (b, L, H).  States
    (b, H, P, N) are ``state_dtype``.  ``fwd`` fills y and final; ``bwd``,
    after a ``fwd`` on the same inputs, dq, dk, dv, dg, dbeta and (with
    initial states) dinit.  The tensors may be refilled between calls.  All are on
    the current CUDA device; the buffers belong to the stream that is current here,
    and calls on another one come after its work."""

    def __init__(self, q, k, v, g, beta, scale=None, initial_states=None, seq_idx=None, dy=None,
                 dfinal_states=None, state_dtype=torch.float32):
        (b, L, H, P, N, G), strides = _delta_shape(q, k, v, g, beta)
        _on_gpu(v.device, "DeltaDevice")
        if state_dtype not in _FLOATS:
            raise ValueError("state_dtype must be fp32 or bf16")
        if dfinal_states is not None and dy is None:
            raise ValueError("dfinal_states needs dy")
        _dense(initial_states, (b, H, P, N), state_dtype, "initial_states", v.device)
        _dense(dfinal_states, (b, H, P, N), state_dtype, "dfinal_states", v.device)
        _dense(seq_idx, (b, L), torch.int32, "seq_idx", v.device)
        _dense(dy, (b, L, H, P), v.dtype, "dy", v.device)
        self.q, self.k, self.v, self.g, self.beta = q, k, v, g, beta
        self.init, self.seq_idx, self.dy, self.dfinal = initial_states, seq_idx, dy, dfinal_states
        dev, dt = v.device, v.dtype
        flags = ((_lib.SSD_HAS_INIT if initial_states is not None else 0)
                 | (_lib.SSD_HAS_SEQ_IDX if seq_idx is not None else 0))
        bflags = flags | (_lib.SSD_HAS_DFINAL if dfinal_states is not None else 0)
        if initial_states is not None:
            bflags |= _lib.SSD_WANT_DINIT
        scale = N ** -0.5 if scale is None else scale
        make = lambda f: _lib.make_delta_problem(  # noqa: E731
            b, L, H, P, N, G, scale, dt, state_dtype, f, *strides)
        self.fwd_prob, self.bwd_prob = make(flags), make(bflags)
        self.y = torch.empty((b, L, H, P), dtype=dt, device=dev)
        self.final = torch.empty((b, H, P, N), dtype=state_dtype, device=dev)
        ws = _lib.ssd_delta_fwd_workspace_bytes(self.fwd_prob)
        if ws == 0:
            raise _lib.SSDError(_lib.SSD_ERR_INVALID_ARGUMENT, "delta workspace size")
        self.saved = None
        if dy is not None:
            ws = max(ws, _lib.ssd_delta_bwd_workspace_bytes(self.bwd_prob))
            self.saved = torch.empty(_lib.ssd_delta_saved_bytes(self.bwd_prob), dtype=torch.uint8,
                                     device=dev)
            self.dq = torch.empty((b, L, G, N), dtype=dt, device=dev)
            self.dk = torch.empty((b, L, G, N), dtype=dt, device=dev)
            self.dv = torch.empty((b, L, H, P), dtype=dt, device=dev)
            self.dg, self.dbeta = torch.empty_like(g), torch.empty_like(beta)
            self.dinit = None if initial_states is None else torch.empty_like(initial_states)
        self.workspace = torch.empty(ws, dtype=torch.uint8, device=dev)

    def fwd(self, stream=None, check=True):
        _on_gpu(self.v.device, "DeltaDevice")
        return _lib.ssd_delta_fwd(self.fwd_prob, self.q, self.k, self.v, self.g, self.beta,
                                  self.init, self.seq_idx, self.y, self.final, self.saved,
                                  self.workspace, stream=stream, check=check)

    def bwd(self, stream=None, check=True):
        if self.saved is None:
            raise ValueError("built without dy: there is no backward")
        _on_gpu(self.v.device, "DeltaDevice")
        return _lib.ssd_delta_bwd(self.bwd_prob, self.q, self.k, self.v, self.g, self.beta,
                                  self.seq_idx, self.dy, self.dfinal, self.dq, self.dk, self.dv,
                                  self.dg, self.dbeta, self.dinit, self.saved, self.workspace,
                                  stream=stream, check=check)

    def device_status(self, stream=None):
        """Synchronises; the status word of the last call."""
        return _lib.ssd_read_device_status(self.workspace, stream)

    def results(self) -> dict:
        out = dict(y=self.y, final_states=self.final)
        if self.dy is not None:
            out.update(dq=self.dq, dk=self.dk, dv=self.dv, dg=self.dg, dbeta=self.dbeta)
            if self.dinit is not None:
                out["dinitial_states"] = self.dinit
        return {k: v.detach().to("cpu", torch.float64) for k, v in out.items()}


class DeltaStepDevice:
    """Token generation with the gated delta rule on a pool of fp32 states
    (nslots, H, P, N).  ``states_out`` defaults to ``states`` (updated in
    place); another pool of the same shape keeps the old ones."""

    def __init__(self, states, states_out=None):
        if states.dim() != 4:
            raise ValueError("states must be (nslots, H, P, N)")
        _on_gpu(states.device, "states")
        _dense(states, states.shape, torch.float32, "states")
        self.states = states
        self.states_out = states if states_out is None else states_out
        _dense(self.states_out, states.shape, torch.float32, "states_out", states.device)

    def step(self, q, k, v, g, beta, scale=None, slots=None, lengths=None, update=True,
             outputs=True, stream=None, check=True):
        """All tokens of q, k (b, T, G, N), v (b, T, H, P), g, beta (b, T, H)
        in order, from each sequence's slot; returns y (b, T, H, P), or None
        without ``outputs`` (y is ``stream``'s: another stream waits for it before
        it reads it).  The states written are those after the first
        ``lengths[b]`` tokens (default: all); ``update=False`` writes none."""
        shape, strides = _delta_shape(q, k, v, g, beta)
        b, T, H, P, N, G = shape
        nslots = self.states.shape[0]
        if self.states.shape[1:] != (H, P, N) or v.device != self.states.device:
            raise ValueError("the tokens' heads do not fit the states")
        _on_gpu(v.device, "DeltaStepDevice")
        _dense(slots, (b,), torch.int32, "slots", v.device)
        _dense(lengths, (b,), torch.int32, "lengths", v.device)
        scale = N ** -0.5 if scale is None else scale
        prob = _step_problem(shape, scale, v.dtype, strides)
        y = None
        if outputs:
            with _allocating_on(stream):
                y = torch.empty((b, T, H, P), dtype=v.dtype, device=v.device)
        _lib.ssd_delta_step(prob, q, k, v, g, beta, nslots, self.states,
                            self.states_out if update else None, slots, lengths, y,
                            stream=stream, check=check)
        return y


def verify_draft(target_probs, draft_probs, draft_tokens, uniform, noise, lengths=None,
                 stream=None, check=True):
    """Keep the drafted tokens that the target accepts and draw the next one:
    (tokens (b, K + 1) int32, kept (b) int32) of target_probs (b, K + 1, V),
    draft_probs (b, K, V) or None, draft_tokens (b, K), uniform (b, K) and
    noise (b, V), standard exponentials.  The results are ``stream``'s: another
    stream waits for it before it reads them."""
    if target_probs.dim() != 3 or target_probs.dtype not in _FLOATS:
        raise ValueError("target_probs must be (b, K + 1, V), fp32 or bf16")
    b, K1, V = target_probs.shape
    dev = target_probs.device
    _on_gpu(dev, "verify_draft")
    _dense(target_probs, (b, K1, V), target_probs.dtype, "target_probs", dev)
    _dense(draft_probs, (b, K1 - 1, V), target_probs.dtype, "draft_probs", dev)
    _dense(draft_tokens, (b, K1 - 1), torch.int32, "draft_tokens", dev)
    _dense(uniform, (b, K1 - 1), torch.float32, "uniform", dev)
    _dense(noise, (b, V), torch.float32, "noise", dev)
    _dense(lengths, (b,), torch.int32, "lengths", dev)
    with _allocating_on(stream):
        tokens = torch.empty((b, K1), dtype=torch.int32, device=dev)
        accepted = torch.empty(b, dtype=torch.int32, device=dev)
    prob = _verify_problem(b, K1 - 1, V, target_probs.dtype)
    _lib.ssd_verify_draft(prob, target_probs, draft_probs, draft_tokens, lengths, uniform, noise,
                          tokens, accepted, stream=stream, check=check)
    return tokens, accepted


class StateCache:
    """An 8-bit cache of recurrent states (nslots, H, P, N): ``int8`` or
    ``e4m3`` values with one fp32 scale for each row of N."""

    FORMATS = {"int8": _lib.SSD_CACHE_INT8, "e4m3": _lib.SSD_CACHE_E4M3}

    def __init__(self, nslots, nheads, headdim, dstate, form="int8", device="cuda"):
        if form not in self.FORMATS:
            raise ValueError(f"form must be one of {sorted(self.FORMATS)}")
        if torch.device(device).type != "cuda":
            raise ValueError(f"the cache lives on a CUDA device, not on {device}")
        self.shape, self.form = (nslots, nheads, headdim, dstate), form
        self.values = torch.empty(self.shape, dtype=torch.uint8, device=device)
        self.scales = torch.zeros(self.shape[:3], dtype=torch.float32, device=device)

    def _prob(self, states, slots):
        b = states.shape[0]
        _on_gpu(self.values.device, "StateCache")
        _dense(states, (b,) + self.shape[1:], torch.float32, "states", self.values.device)
        _dense(slots, (b,), torch.int32, "slots", self.values.device)
        return _cache_problem(b, *self.shape[1:], self.shape[0], self.FORMATS[self.form])

    def store(self, states, slots=None, stream=None, check=True):
        """Quantise states (b, H, P, N) into their slots (default: 0 .. b-1)."""
        return _lib.ssd_state_cache_store(self._prob(states, slots), states, slots, self.values,
                                          self.scales, stream=stream, check=check)

    def load(self, slots, out, stream=None, check=True):
        """Read the slots' states (None: 0 .. b-1) into out (b, H, P, N); a
        slot may be read many times, one outside the cache gives zeros."""
        return _lib.ssd_state_cache_load(self._prob(out, slots), self.values, self.scales, slots,
                                         out, stream=stream, check=check)
