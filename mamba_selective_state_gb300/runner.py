"""Device buffers for one SSD problem and the calls that run it through the
C ABI.  Allocation and argument marshalling only; the layer runs in libssd.
"""
from __future__ import annotations

import contextlib
import ctypes
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


def _here(device, what, stream):
    """The stream's handle for a call of a single token's size, after _on_gpu's
    check of the tensors' device."""
    if torch.cuda.current_device() != device.index:
        _on_gpu(device, what)
    if stream is None and _lib._raw_stream is not None:
        return _lib._raw_stream(device.index)
    return _lib._stream(stream)


def _raise(rc, check, what):
    if check and rc != _lib.SSD_OK:
        raise _lib.SSDError(rc, what)
    return rc


# torch's types of the 8-bit codes
CODE_TYPES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


class AddNormDevice:
    """The norm that takes in the residual: the caller's device tensors, the
    outputs and the calls through the C ABI.

    x (rows, dim), rows evenly spaced; residual (rows, dim), x's type or fp32,
    or None.  ``fwd`` fills h (residual's type; x itself without a residual) and
    out, or with ``form`` ("int8", "e4m3") codes and scales; ``h_out`` (the
    residual itself, for instance) takes h instead of a buffer of its own.
    With ``dout`` (x's type) and optionally ``dh`` (h's), ``bwd`` after a ``fwd``
    fills dx, dresidual (dx itself where the types are the same) and dweight.
    The tensors may be refilled between calls.  All are on the current CUDA
    device; the buffers belong to the stream that is current here, and calls on
    another one come after its work."""

    FORMATS = {None: _lib.SSD_OUT_PLAIN, "int8": _lib.SSD_OUT_INT8, "e4m3": _lib.SSD_OUT_E4M3}

    def __init__(self, x, weight, residual=None, eps=1e-5, form=None, h_out=None, dout=None,
                 dh=None):
        if x.dim() != 2 or x.dtype not in _FLOATS:
            raise ValueError("x must be (rows, dim), fp32 or bf16")
        if form not in self.FORMATS:
            raise ValueError("form must be None, 'int8' or 'e4m3'")
        rows, dim = x.shape
        dev = x.device
        stride = x.stride(0) if rows > 1 else dim
        if (dim > 1 and x.stride(1) != 1) or stride < dim:
            raise ValueError("x: its rows must be dense and evenly spaced")
        rt = x.dtype if residual is None else residual.dtype
        if rt is not x.dtype and rt is not torch.float32:
            raise ValueError("residual must be of x's type or fp32")
        _on_gpu(dev, "AddNormDevice")
        _dense(weight, (dim,), torch.float32, "weight", dev)
        _dense(residual, (rows, dim), rt, "residual", dev)
        _dense(h_out, (rows, dim), rt, "h_out", dev)
        _dense(dout, (rows, dim), x.dtype, "dout", dev)
        _dense(dh, (rows, dim), rt, "dh", dev)
        if dh is not None and dout is None:
            raise ValueError("dh needs dout")
        if residual is None and h_out is None and dout is not None and not x.is_contiguous():
            raise ValueError("the backward reads x as h: it must be dense")
        self.x, self.weight, self.residual, self.dout, self.dh = x, weight, residual, dout, dh
        self.prob = _lib.make_add_norm_problem(rows, dim, eps, x.dtype, rt, self.FORMATS[form],
                                               residual is not None, stride)
        self._ref = ctypes.byref(self.prob)
        ws = _lib.ssd_add_rmsnorm_bwd_workspace_bytes(self.prob)
        if ws == 0:
            raise _lib.SSDError(_lib.SSD_ERR_INVALID_ARGUMENT, "add_norm problem")
        new = lambda dt: torch.empty((rows, dim), dtype=dt, device=dev)  # noqa: E731
        self.out = self.codes = self.scales = None
        if form is None:
            self.out = new(x.dtype)
        else:
            self.codes = new(CODE_TYPES[form])
            self.scales = torch.empty(rows, dtype=torch.float32, device=dev)
        self._h = h_out if h_out is not None else None if residual is None else new(rt)
        self.h = x if self._h is None else self._h
        if dout is not None:
            self.dx = new(x.dtype)
            self.dresidual = None if residual is None else self.dx if rt is x.dtype else new(rt)
            self.dweight = torch.empty(dim, dtype=torch.float32, device=dev)
            self.workspace = torch.empty(ws, dtype=torch.uint8, device=dev)

    def fwd(self, stream=None, check=True):
        handle = _here(self.x.device, "AddNormDevice", stream)
        out, p = self.codes if self.out is None else self.out, _lib._p
        rc = _lib.LIB.ssd_add_rmsnorm_fwd(self._ref, self.x.data_ptr(), p(self.residual),
                                          self.weight.data_ptr(), p(self._h), out.data_ptr(),
                                          p(self.scales), handle)
        return _raise(rc, check, "ssd_add_rmsnorm_fwd")

    def bwd(self, stream=None, check=True):
        if self.dout is None:
            raise ValueError("built without dout: there is no backward")
        handle, p = _here(self.x.device, "AddNormDevice", stream), _lib._p
        own = None if self.dresidual is self.dx else self.dresidual
        rc = _lib.LIB.ssd_add_rmsnorm_bwd(self._ref, self.h.data_ptr(), self.weight.data_ptr(),
                                          self.dout.data_ptr(), p(self.dh), self.dx.data_ptr(),
                                          p(own), self.dweight.data_ptr(),
                                          self.workspace.data_ptr(), self.workspace.numel(), handle)
        return _raise(rc, check, "ssd_add_rmsnorm_bwd")


class Linear8:
    """A linear map whose weights are 8-bit codes (n, k), int8 or e4m3, with a
    scale for each output channel; it takes tokens in the same codes with a
    scale for each, as AddNormDevice writes them."""

    def __init__(self, codes, scales, bias=None, out_dtype=torch.bfloat16):
        if codes.dim() != 2 or codes.dtype not in CODE_TYPES.values():
            raise ValueError("codes must be (n, k), int8 or float8_e4m3fn")
        if out_dtype not in _FLOATS:
            raise ValueError("out_dtype must be fp32 or bf16")
        n = codes.shape[0]
        _on_gpu(codes.device, "Linear8")
        _dense(codes, codes.shape, codes.dtype, "codes", codes.device)
        _dense(scales, (n,), torch.float32, "scales", codes.device)
        _dense(bias, (n,), torch.float32, "bias", codes.device)
        self.codes, self.scales, self.bias, self.out_dtype = codes, scales, bias, out_dtype
        self.format = StateCache.FORMATS["int8" if codes.dtype is torch.int8 else "e4m3"]
        self._plans = {}
        # the status words of calls that need no more: one to a stream, whose calls follow one another
        self._words = {}
        self.workspace = torch.zeros(256, dtype=torch.uint8, device=codes.device)
        self._last = None       # the stream's handle of the last call

    @classmethod
    def from_weight(cls, weight, form="int8", bias=None, out_dtype=torch.bfloat16):
        """Weights (n, k) rounded to 8 bits, a scale for each row of k: by the
        state cache's rule, once."""
        if form not in CODE_TYPES:
            raise ValueError(f"form must be one of {sorted(CODE_TYPES)}")
        if weight.dim() != 2 or weight.numel() == 0:
            raise ValueError("weight must be (n, k)")
        w = weight.detach().float().contiguous()
        top = 127.0 if form == "int8" else 448.0
        big = w.abs().amax(1, keepdim=True)
        bad = ~torch.isfinite(w).all(1, keepdim=True)
        empty = ~(big >= 2.0 ** -118)
        y = torch.where(bad | empty, 0.0, w * torch.where(empty, 0.0, (1.0 / big) * top))
        y = torch.round(y).clamp_(-127, 127) if form == "int8" else y.clamp_(-448, 448)
        scales = torch.where(bad, float("nan"), torch.where(empty, 0.0, big * (1.0 / top)))
        return cls(y.to(CODE_TYPES[form]), scales[:, 0].contiguous(), bias, out_dtype)

    def __call__(self, codes, scales, out=None, stream=None, check=True):
        """out (m, n) of the tokens' codes (m, k) and scales (m); a new tensor
        unless given (``stream``'s: another stream waits for it before it reads
        it)."""
        plan = self._plans.get(codes.shape) or self._plan(codes.shape)
        prob, ws, scales_shape, out_shape = plan
        dev, index = self.codes.device, self.codes.get_device()
        handle = _here(dev, "Linear8", stream)
        # (single tokens: these comparisons are the cheap ones)
        if codes.dtype is not self.codes.dtype or codes.get_device() != index or not codes.is_contiguous():
            _dense(codes, codes.shape, self.codes.dtype, "codes", dev)
        if (scales.dtype is not torch.float32 or scales.get_device() != index or scales.shape != scales_shape
                or not scales.is_contiguous()):
            _dense(scales, scales_shape, torch.float32, "scales", dev)
        if out is None:
            if stream is None:
                out = torch.empty(out_shape, dtype=self.out_dtype, device=dev)
            else:
                with _allocating_on(stream):
                    out = torch.empty(out_shape, dtype=self.out_dtype, device=dev)
        else:
            _dense(out, out_shape, self.out_dtype, "out", dev)
        # a call that is being captured (never on the default stream) has its own memory: graphs may be replayed side by side
        own = ws or (handle and torch.cuda.is_current_stream_capturing())
        work = None if own else self._words.get(handle)
        if work is None:
            with _allocating_on(stream):
                work = torch.empty(ws or 256, dtype=torch.uint8, device=dev)
            if not own:
                self._words[handle] = work
        rc = _lib.LIB.ssd_scaled_matmul(ctypes.byref(prob), codes.data_ptr(), scales.data_ptr(),
                                        self.codes.data_ptr(), self.scales.data_ptr(),
                                        _lib._p(self.bias), out.data_ptr(), work.data_ptr(),
                                        ws or 256, handle)
        self.workspace, self._last = work, handle
        _raise(rc, check, "ssd_scaled_matmul")
        return out

    def _plan(self, shape):
        """The problem of tokens (m, k), the bytes of its workspace where it needs
        more than the status word, and its tensors' shapes; kept for shapes that
        come again."""
        n, k = self.codes.shape
        if len(shape) != 2 or shape[1] != k:
            raise ValueError(f"codes: expected (m, {k})")
        prob = _lib.make_matmul_problem(shape[0], n, k, self.format, self.out_dtype)
        ws = _lib.ssd_scaled_matmul_workspace_bytes(prob)
        if ws == 0:
            raise _lib.SSDError(_lib.SSD_ERR_INVALID_ARGUMENT, "matmul problem")
        if len(self._plans) >= 256:
            self._plans.clear()
        self._plans[shape] = plan = (prob, ws if ws > 256 else 0, torch.Size(shape[:1]), (shape[0], n))
        return plan

    def device_status(self, stream=None):
        """The status word of the last call, behind that call -- or behind
        ``stream``'s work, where a graph that holds the call was replayed there."""
        if stream is None and self._last not in (None, _here(self.codes.device, "Linear8", None)):
            torch.cuda.synchronize(self.codes.device)
        return _lib.ssd_read_device_status(self.workspace, stream)


class LogProbsDevice:
    """Log probabilities of given tokens: the caller's device tensors, the
    outputs and the calls through the C ABI.

    logits (rows, vocab), fp32 or bf16, rows evenly spaced; tokens (rows) int32
    (outside the vocabulary: padding).  Tensors begin on 16-byte boundaries
    (clone a slice such as ``tokens[1:]``).  ``fwd`` fills logprobs, entropy, lse
    (rows) and, with ``ntop``, top_tokens and top_logprobs (rows, ntop).  With
    ``dlogprobs`` and/or ``dentropy`` (rows), ``bwd`` after a ``fwd`` fills
    dlogits, laid out as logits; ``dlogits=logits`` overwrites them.  A row of
    padding whose dentropy is 0 or not given gets zeros, whatever its logits hold.
    The tensors may be refilled between calls.  All are on the current CUDA device; the
    buffers belong to the stream that is current here, and calls on another one
    come after its work."""

    def __init__(self, logits, tokens, scale=1.0, ntop=0, dlogprobs=None, dentropy=None,
                 dlogits=None):
        if logits.dim() != 2 or logits.dtype not in _FLOATS:
            raise ValueError("logits must be (rows, vocab), fp32 or bf16")
        rows, vocab = logits.shape
        dev = logits.device
        spaced = lambda t: t.stride(0) if rows > 1 else vocab  # noqa: E731
        for t, what in ((logits, "logits"), (dlogits, "dlogits")):
            if t is not None and (t.shape != logits.shape or t.dtype is not logits.dtype or t.device != dev
                                  or (vocab > 1 and t.stride(1) != 1) or spaced(t) < vocab):
                raise ValueError(f"{what}: expected (rows, vocab) with dense, evenly spaced rows")
        _on_gpu(dev, "LogProbsDevice")
        _dense(tokens, (rows,), torch.int32, "tokens", dev)
        _dense(dlogprobs, (rows,), torch.float32, "dlogprobs", dev)
        _dense(dentropy, (rows,), torch.float32, "dentropy", dev)
        self.back = dlogprobs is not None or dentropy is not None
        if dlogits is not None and not self.back:
            raise ValueError("dlogits needs dlogprobs or dentropy")
        self.logits, self.tokens, self.dlogprobs, self.dentropy = logits, tokens, dlogprobs, dentropy
        self.dlogits = dlogits
        if self.back and dlogits is None:
            self.dlogits = torch.empty((rows, vocab), dtype=logits.dtype, device=dev)
        self.prob = _lib.make_logprob_problem(rows, vocab, scale, ntop, logits.dtype, spaced(logits),
                                              spaced(self.dlogits) if self.back else 0)
        self._ref = ctypes.byref(self.prob)
        new = lambda *s, dt=torch.float32: torch.empty(s, dtype=dt, device=dev)  # noqa: E731
        self.logprobs, self.entropy, self.lse = new(rows), new(rows), new(rows)
        self.stats = new(rows, 2) if self.back else None
        self.top_tokens = new(rows, ntop, dt=torch.int32) if ntop else None
        self.top_logprobs = new(rows, ntop) if ntop else None

    def fwd(self, stream=None, check=True):
        handle, p = _here(self.logits.device, "LogProbsDevice", stream), _lib._p
        rc = _lib.LIB.ssd_token_logprobs(self._ref, self.logits.data_ptr(), self.tokens.data_ptr(),
                                         self.logprobs.data_ptr(), self.entropy.data_ptr(),
                                         self.lse.data_ptr(), p(self.stats), p(self.top_tokens),
                                         p(self.top_logprobs), handle)
        return _raise(rc, check, "ssd_token_logprobs")

    def bwd(self, stream=None, check=True):
        if not self.back:
            raise ValueError("built without dlogprobs and dentropy: there is no backward")
        handle, p = _here(self.logits.device, "LogProbsDevice", stream), _lib._p
        rc = _lib.LIB.ssd_token_logprobs_bwd(
            self._ref, self.logits.data_ptr(), None if self.dlogprobs is None else self.tokens.data_ptr(),
            self.stats.data_ptr(), None if self.dentropy is None else self.entropy.data_ptr(),
            p(self.dlogprobs), p(self.dentropy), self.dlogits.data_ptr(), handle)
        return _raise(rc, check, "ssd_token_logprobs_bwd")
