"""Device buffers for one call of each fused operator, and the call itself.

Owns the plumbing around an entry point -- uploading the seeded inputs,
allocating the receive windows, flag arrays, workspace and status word with
PyTorch, advancing the epoch -- so that tests, the bench and the smoke check
drive the C ABI the same way.  No arithmetic of the operators lives here.
bf16 tensors are carried as ``torch.int16`` (their bit patterns).
"""

from __future__ import annotations

import numpy as np
import torch

from . import hocf

F32, BF16 = hocf.HOCF_F32, hocf.HOCF_BF16


def tdtype(dt):
    return torch.int16 if dt == BF16 else torch.float32


def to_device(a: np.ndarray, device="cuda") -> torch.Tensor:
    if a.dtype == np.uint16:
        a = a.view(np.int16)
    return torch.from_numpy(np.ascontiguousarray(a)).to(device)


def to_host(t: torch.Tensor, dt) -> np.ndarray:
    a = t.detach().cpu().numpy()
    return a.view(np.uint16) if dt == BF16 else a


def nan_fill(t: torch.Tensor) -> None:
    """Poison a buffer so that any element the kernel does not write shows up."""
    if t.dtype == torch.int16:
        t.fill_(0x7FC0)          # bf16 quiet NaN
    elif t.dtype == torch.float32:
        t.fill_(float("nan"))
    else:
        t.fill_(-1)


def cdiv(a, b):
    return (a + b - 1) // b


class _Common:
    def _alloc_sync(self, ws_bytes, device):
        self.ws_bytes = max(int(ws_bytes), 16)
        self.ws = torch.zeros(cdiv(self.ws_bytes, 4) + 4, dtype=torch.int32, device=device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self.epoch = 0

    def next_sync(self, spin_timeout_ns=0, abort_flag=None):
        self.epoch = (self.epoch % 0xFFFFFFF0) + 1
        return hocf.sync(self.epoch, self.ws, self.ws_bytes, status=self.status,
                         abort_flag=abort_flag, spin_timeout_ns=spin_timeout_ns)

    def status_value(self) -> int:
        return int(self.status.item())

    def report_to(self, word: torch.Tensor) -> None:
        """What later calls report asynchronously goes to this status word (int32 [1])."""
        self.status = word


class GemmRS(_Common):
    """hocf_gemm_rs: A [P][M][K], W [P][K][N] -> windows [P dst][P src][Mc][N], out [M][N]."""

    def __init__(self, P, M, N, K, in_dt, slot_dt, out_dt, tile_m, tile_n, A, W, device="cuda",
                 unfused=False, noalloc=False, pieces=0, fold_cus=0):
        self.unfused = unfused   # hocf_gemm_rs_unfused: the GEMM kernel, then the fold kernel
        self.noalloc = noalloc   # hocf_gemm_rs_noalloc: no workspace (the library's scratch)
        # hocf_gemm_rs_decomposed: `pieces` column pieces, GEMM on the call's stream (leaving
        # fold_cus CUs), each fold on a second stream
        self.pieces, self.fold_cus = pieces, fold_cus
        self.coll = torch.cuda.Stream(device=device) if pieces else None
        self.P, self.M, self.N, self.K = P, M, N, K
        self.in_dt, self.slot_dt, self.out_dt = in_dt, slot_dt, out_dt
        self.tile_m, self.tile_n = tile_m, tile_n
        self.Mc = M // P
        self.A = A if isinstance(A, torch.Tensor) else to_device(A, device)
        self.W = W if isinstance(W, torch.Tensor) else to_device(W, device)
        self.tpc = cdiv(self.Mc, tile_m) * cdiv(N, tile_n)
        self.win_data = torch.empty((P, P, self.Mc, N), dtype=tdtype(slot_dt), device=device)
        self.win_flags = torch.zeros((P, P, self.tpc), dtype=torch.int32, device=device)
        self.out = torch.empty((M, N), dtype=tdtype(out_dt), device=device)
        self.win = hocf.windows([(self.win_data[r], self.win_flags[r]) for r in range(P)])
        self._alloc_sync(hocf.hocf_gemm_rs_workspace_bytes(P, M, N, tile_m, tile_n), device)

    def poison(self):
        nan_fill(self.win_data)
        nan_fill(self.out)

    def call(self, stream=None, **kw) -> int:
        s = self.next_sync(**kw)
        if getattr(self, "pieces", 0):
            return hocf.hocf_gemm_rs_decomposed(self.P, self.M, self.N, self.K, self.in_dt, self.slot_dt,
                                                self.out_dt, self.A, self.W, self.win, self.out, self.tile_m,
                                                self.tile_n, self.pieces, self.fold_cus, s,
                                                stream if stream is not None else torch.cuda.current_stream(),
                                                self.coll)
        if getattr(self, "noalloc", False):
            s.workspace, s.workspace_bytes = None, 0
            fn = hocf.hocf_gemm_rs_noalloc
        else:
            fn = hocf.hocf_gemm_rs_unfused if self.unfused else hocf.hocf_gemm_rs
        return fn(self.P, self.M, self.N, self.K, self.in_dt, self.slot_dt, self.out_dt, self.A, self.W,
                  self.win, self.out, self.tile_m, self.tile_n, s, stream)

    def run(self, stream=None, **kw):
        hocf.check(self.call(stream, **kw))


class GemmAR(GemmRS):
    """hocf_gemm_ar: as GemmRS, and every destination q gets the whole reduced
    result in outs[q] = [M][N] (held together as out_all [P][M][N])."""

    def __init__(self, P, M, N, K, in_dt, slot_dt, out_dt, tile_m, tile_n, A, W, device="cuda"):
        super().__init__(P, M, N, K, in_dt, slot_dt, out_dt, tile_m, tile_n, A, W, device)
        del self.unfused
        del self.out
        self.out_all = torch.empty((P, M, N), dtype=tdtype(out_dt), device=device)
        self.outs = hocf.pointers([self.out_all[q] for q in range(P)])

    def poison(self):
        nan_fill(self.win_data)
        nan_fill(self.out_all)

    def call(self, stream=None, **kw) -> int:
        s = self.next_sync(**kw)
        return hocf.hocf_gemm_ar(self.P, self.M, self.N, self.K, self.in_dt, self.slot_dt,
                                 self.out_dt, self.A, self.W, self.win, self.outs, self.tile_m,
                                 self.tile_n, s, stream)


class GemvAR(_Common):
    """hocf_gemv_ar: x [P][Mb][K], W [P][K][N] -> part [P][Mb][N], windows [P][Mb][N]."""

    def __init__(self, P, Mb, N, K, in_dt, slot_dt, out_dt, tile_n, x, W, device="cuda", unfused=False):
        self.unfused = unfused   # hocf_gemv_ar_unfused: the GEMV kernel, then the fold kernel
        self.P, self.Mb, self.N, self.K = P, Mb, N, K
        self.in_dt, self.slot_dt, self.out_dt, self.tile_n = in_dt, slot_dt, out_dt, tile_n
        self.x = x if isinstance(x, torch.Tensor) else to_device(x, device)
        self.W = W if isinstance(W, torch.Tensor) else to_device(W, device)
        self.nt = cdiv(N, tile_n)
        self.part = torch.empty((P, Mb, N), dtype=tdtype(slot_dt), device=device)
        self.part_flags = torch.zeros((P, self.nt), dtype=torch.int32, device=device)
        self.win_data = torch.empty((P, Mb, N), dtype=tdtype(out_dt), device=device)
        self.win_flags = torch.zeros((P, self.nt), dtype=torch.int32, device=device)
        self.win = hocf.windows([(self.win_data[q], self.win_flags[q]) for q in range(P)])
        self._alloc_sync(hocf.hocf_gemv_ar_workspace_bytes(P, N, tile_n), device)

    def set_weights(self, x, W):
        self.x, self.W = x, W

    def poison(self):
        nan_fill(self.part)
        nan_fill(self.win_data)

    def call(self, stream=None, **kw) -> int:
        s = self.next_sync(**kw)
        fn = hocf.hocf_gemv_ar_unfused if self.unfused else hocf.hocf_gemv_ar
        return fn(self.P, self.Mb, self.N, self.K, self.in_dt, self.slot_dt, self.out_dt, self.x, self.W,
                  self.part, self.part_flags, self.win, self.tile_n, s, stream)

    def run(self, stream=None, **kw):
        hocf.check(self.call(stream, **kw))


class AgGemm(_Common):
    """hocf_ag_gemm: gathered chunks [P][Mc][K] gated by chunk_flags [P]; W [K][N] -> out.

    flags="device": chunk flags in device memory, written on the kernel's own
    stream before the kernel (all chunks present when it starts).
    flags="host": chunk flags in coherent pinned host memory, written by the
    host while the kernel runs (paced, any order, or withheld).
    chunks_on_host: the gathered chunks themselves live in coherent pinned host
    memory too, so the host can deliver them after the kernel has started."""

    def __init__(self, P, Mc, N, K, out_dt, tile_m, tile_n, chunks, W, device="cuda",
                 flags="device", chunks_on_host=False):
        self.P, self.Mc, self.N, self.K = P, Mc, N, K
        self.out_dt, self.tile_m, self.tile_n = out_dt, tile_m, tile_n
        self.flags_mode = flags
        self.W = W if isinstance(W, torch.Tensor) else to_device(W, device)
        self.host_chunks = None
        if chunks_on_host:
            nbytes = P * Mc * K * 2
            addr, _ = hocf.host_coherent(nbytes)
            self.A = addr
            self.host_chunks = np.frombuffer((ctypes_char_array(addr, nbytes)), dtype=np.uint16).reshape(P, Mc, K)
        else:
            self.A = chunks if isinstance(chunks, torch.Tensor) else to_device(chunks, device)
        if flags == "host":
            addr, _ = hocf.host_coherent(4 * P)
            self.chunk_flags = addr
            self.host_flags = np.frombuffer(ctypes_char_array(addr, 4 * P), dtype=np.uint32)
        else:
            self.chunk_flags = torch.zeros(P, dtype=torch.int32, device=device)
            self.host_flags = None
        self.out = torch.empty((P * Mc, N), dtype=tdtype(out_dt), device=device)
        self._alloc_sync(hocf.hocf_ag_gemm_workspace_bytes(P), device)

    def poison(self):
        nan_fill(self.out)

    def call(self, sync_, stream=None) -> int:
        return hocf.hocf_ag_gemm(self.P, self.Mc, self.N, self.K, BF16, self.out_dt, self.A,
                                 self.chunk_flags, self.W, self.out, self.tile_m, self.tile_n,
                                 sync_, stream)

    def prerelease(self, order, stream=None, **kw):
        """Writes the chunk flags in `order` on `stream` for the next call; returns its sync."""
        assert self.flags_mode == "device"
        s = self.next_sync(**kw)
        hocf.release_chunks(stream or torch.cuda.current_stream(), self.chunk_flags, order, s.epoch)
        return s

    def launch(self, sync_, stream=None):
        hocf.check(self.call(sync_, stream or torch.cuda.current_stream()))

    def run_prereleased(self, order, stream=None, **kw):
        """Flags written in `order` on the kernel's stream, then the kernel."""
        stream = stream or torch.cuda.current_stream()
        self.launch(self.prerelease(order, stream, **kw), stream)

    def run_host_released(self, order, delay_s=0.0, deliver=None, stream=None, **kw):
        """Kernel first; then the host sets the flags of `order` one by one (after
        `delay_s` each), optionally delivering chunk c's data first via deliver(c)."""
        import time
        assert self.flags_mode == "host"
        s = self.next_sync(**kw)
        stream = stream or torch.cuda.current_stream()
        hocf.check(self.call(s, stream))
        for c in order:
            if delay_s:
                time.sleep(delay_s)
            if deliver is not None:
                deliver(int(c))
            self.host_flags[int(c)] = s.epoch
        return s.epoch


    def put_delivered(self, sources, order, engine, put_stream, stream=None, **kw):
        """Chunks delivered by hocf_dma_put on `put_stream` while the kernel runs on
        `stream`: one put per chunk in `order` (chunk c's bytes from sources[c] into
        its rows of the gathered buffer, then its flag); sources[c] None: the chunk is
        already in place (the local one) and its put only signals.  The puts are
        enqueued first and wait for nothing but `stream`'s earlier work, so the
        kernel starts while they land.  Returns the call's sync."""
        assert self.flags_mode == "device" and isinstance(self.A, torch.Tensor)
        stream = stream or torch.cuda.current_stream()
        s = self.next_sync(**kw)
        if s.epoch >= _EPOCH_WORDS:
            # the signal table holds epochs below 2^16: start over at 1 (it still
            # differs from the previous call's epoch, the flags' only requirement)
            self.epoch = 0
            s = self.next_sync(**kw)
        chunk_bytes = self.Mc * self.K * 2
        base, fbase = self.A.data_ptr(), self.chunk_flags.data_ptr()
        src, dst, nbytes, sig = [], [], [], []
        for c in order:
            c = int(c)
            here = sources[c] is None
            src.append(None if here else sources[c])
            dst.append(None if here else base + c * chunk_bytes)
            nbytes.append(0 if here else chunk_bytes)
            sig.append(fbase + 4 * c)
        put_stream.wait_stream(stream)
        hocf.check(hocf.hocf_dma_put(src, dst, nbytes, sig, epoch_word(s.epoch, self.A.device), engine,
                                     put_stream))
        hocf.check(self.call(s, stream))
        stream.wait_stream(put_stream)
        return s


_epoch_words = {}
_EPOCH_WORDS = 1 << 16


def epoch_word(epoch: int, device) -> int:
    """Device address of a word holding `epoch` (1 <= epoch < 65536), from a table
    written once per device: the source a put copies into a flag, so that the
    put's signal needs no kernel to prepare it."""
    assert 1 <= epoch < _EPOCH_WORDS, epoch
    key = str(device)
    if key not in _epoch_words:
        _epoch_words[key] = torch.arange(_EPOCH_WORDS, dtype=torch.int32, device=device)
        torch.cuda.synchronize(device)
    return _epoch_words[key].data_ptr() + 4 * epoch


def ctypes_char_array(addr, nbytes):
    import ctypes
    return (ctypes.c_char * nbytes).from_address(addr)


class EmbbagA2A(_Common):
    """hocf_embbag_a2a: tables [T][R][D], indices -> windows [P][Bd][T][D]."""

    def __init__(self, T, R, D, B, L, P, tile_bags, tables, indices, offsets=None, device="cuda"):
        self.T, self.R, self.D, self.B, self.L, self.P = T, R, D, B, L, P
        self.tile_bags = tile_bags
        self.Bd = B // P
        self.nj = cdiv(self.Bd, tile_bags)
        self.tables = tables if isinstance(tables, torch.Tensor) else to_device(tables, device)
        self.indices = indices if isinstance(indices, torch.Tensor) else to_device(indices, device)
        self.offsets = None
        if offsets is not None:
            self.offsets = offsets if isinstance(offsets, torch.Tensor) else to_device(offsets, device)
        self.win_data = torch.empty((P, self.Bd, T, D), dtype=torch.float32, device=device)
        self.win_flags = torch.zeros((P, T, self.nj), dtype=torch.int32, device=device)
        self.win = hocf.windows([(self.win_data[d], self.win_flags[d]) for d in range(P)])
        self._alloc_sync(hocf.hocf_embbag_a2a_workspace_bytes(), device)

    def poison(self):
        nan_fill(self.win_data)

    def call(self, stream=None, **kw) -> int:
        s = self.next_sync(**kw)
        return hocf.hocf_embbag_a2a(self.T, self.R, self.D, self.B, 0 if self.offsets is not None else self.L,
                                    self.P, self.tables, self.indices, self.offsets, self.win,
                                    self.tile_bags, s, stream)

    def run(self, stream=None, **kw):
        hocf.check(self.call(stream, **kw))


class GemmA2A(_Common):
    """hocf_gemm_a2a: X [T][K] grouped by expert (offsets), W [E][K][N], routing
    dest/slot [T] -> windows [P][cap][N] with one flag word each."""

    def __init__(self, P, E, N, K, out_dt, X, W, offsets, dest, slot, send_counts, cap, device="cuda",
                 tile_m=256):
        self.P, self.E, self.N, self.K, self.out_dt, self.cap = P, E, N, K, out_dt, cap
        self.tile_m = tile_m
        self.offsets = np.ascontiguousarray(offsets, dtype=np.int64)
        self.send_counts = np.ascontiguousarray(send_counts, dtype=np.int64)
        self.T = int(self.offsets[-1])
        self.X = X if isinstance(X, torch.Tensor) else to_device(X, device)
        self.W = W if isinstance(W, torch.Tensor) else to_device(W, device)
        self.dest = to_device(np.ascontiguousarray(dest, dtype=np.int32), device)
        self.slot = to_device(np.ascontiguousarray(slot, dtype=np.int32), device)
        self.win_data = torch.empty((P, cap, N), dtype=tdtype(out_dt), device=device)
        self.win_flags = torch.zeros((P, 4), dtype=torch.int32, device=device)  # word 0 used; 16-byte rows
        self.win = hocf.windows([(self.win_data[d], self.win_flags[d]) for d in range(P)])
        self._alloc_sync(hocf.hocf_gemm_a2a_workspace_bytes(P), device)

    def poison(self):
        nan_fill(self.win_data)

    def call(self, stream=None, **kw) -> int:
        s = self.next_sync(**kw)
        return hocf.hocf_gemm_a2a(self.P, self.E, self.T, self.N, self.K, BF16, self.out_dt, self.X, self.W,
                                  self.offsets, self.dest, self.slot, self.send_counts, self.win, self.cap,
                                  self.tile_m, 256, s, stream)

    def run(self, stream=None, **kw):
        hocf.check(self.call(stream, **kw))


class A2aGemm(_Common):
    """hocf_a2a_gemm: token rows X [P][B][K] and router choices [P][B][topk] of the
    P source ranks, this rank's experts W [E][K][N] (global ids e0 ..) -> the
    received rows recv [cap][K] grouped by expert, Y [cap][N], expert_offsets
    [E+1], dest / slot [cap], send_counts [P]."""

    def __init__(self, P, E, e0, B, topk, N, K, out_dt, X, experts, W, cap, tile_m=256, device="cuda",
                 unfused=False):
        self.P, self.E, self.e0, self.B, self.topk, self.N, self.K = P, E, e0, B, topk, N, K
        self.out_dt, self.cap, self.tile_m, self.unfused = out_dt, cap, tile_m, unfused
        self.X = X if isinstance(X, torch.Tensor) else to_device(X, device)
        self.W = W if isinstance(W, torch.Tensor) else to_device(W, device)
        self.experts = experts if isinstance(experts, torch.Tensor) else \
            to_device(np.ascontiguousarray(experts, dtype=np.int32), device)
        self.recv = torch.empty((cap, K), dtype=torch.int16, device=device)
        self.Y = torch.empty((cap, N), dtype=tdtype(out_dt), device=device)
        self.offsets = torch.empty(E + 1, dtype=torch.int64, device=device)
        self.dest = torch.empty(cap, dtype=torch.int32, device=device)
        self.slot = torch.empty(cap, dtype=torch.int32, device=device)
        self.send_counts = torch.empty(P, dtype=torch.int64, device=device)
        self._alloc_sync(hocf.hocf_a2a_gemm_workspace_bytes(P, E, B, topk, cap, tile_m), device)

    def poison(self):
        nan_fill(self.recv)
        nan_fill(self.Y)
        self.dest.fill_(-77)        # (not -1: that is what padding rows get)
        self.slot.fill_(-77)
        self.offsets.fill_(-7)
        self.send_counts.fill_(-7)

    def call(self, stream=None, **kw) -> int:
        s = self.next_sync(**kw)
        return hocf.hocf_a2a_gemm(self.P, self.E, self.e0, self.B, self.topk, self.N, self.K, BF16, self.out_dt,
                                  self.X, self.experts, self.W, self.cap, self.recv, self.Y, self.offsets,
                                  self.dest, self.slot, self.send_counts, self.tile_m, 256, s, stream,
                                  unfused=self.unfused)

    def run(self, stream=None, **kw):
        hocf.check(self.call(stream, **kw))


def torch_dt(t: torch.Tensor) -> int:
    """The library's type of a tensor (bf16 as torch.bfloat16 or as its bit patterns)."""
    if t.dtype in (torch.bfloat16, torch.int16):
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"{t.dtype}: the library takes fp32 and bf16")


def _on(device, **tensors):
    """Raises unless `device` is a GPU and every tensor given is on it."""
    if device.type != "cuda":
        raise ValueError(f"the tensors are on {device}: the operators take a GPU's memory")
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, not on {device}")


def _dense(dtype, shape, **tensors):
    """Raises unless every tensor given has this dtype and shape, dense and row-major."""
    for name, t in tensors.items():
        if t is None:
            continue
        if dtype is not None and t.dtype != dtype:
            raise TypeError(f"{name} is {t.dtype}, not {dtype}")
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name} is not contiguous")


class _Moe(_Common):
    """What the mixture-of-experts operators share: inputs are torch tensors, used
    where they are (no copy); a call goes to the current stream of their device
    unless it is given one.  A handle makes its outputs and workspace on the current
    stream and reads and writes the same memory at every call: calls on another
    stream are ordered behind that, and the handle is kept until they have ended."""

    def _bind(self, entry, args, device, ws_bytes=0):
        self._alloc_sync(ws_bytes, device)
        self._sync = self.next_sync()
        self._fn = hocf.bind(entry, args, self._sync)
        self._index = torch.cuda.current_device() if device.index is None else device.index

    def report_to(self, word):
        super().report_to(word)
        self._sync.status = word.data_ptr()

    def call(self, stream=None) -> int:
        self.epoch = self._sync.epoch = (self.epoch % 0xFFFFFFF0) + 1
        return self._fn(torch._C._cuda_getCurrentRawStream(self._index) if stream is None else hocf._stream(stream))

    def run(self, stream=None):
        hocf.check(self.call(stream))


def _rows_ld(logits, T, E):
    """Row stride of the logits: [T][E], the experts of a row adjacent, the rows E or more
    apart (the kernels read E logits from every row's start: rows that share memory, as an
    expanded tensor's do, would be read beyond their end)."""
    if tuple(logits.shape) != (T, E):
        raise ValueError(f"logits have shape {tuple(logits.shape)}, not {(T, E)}")
    if E > 1 and logits.stride(1) != 1:
        raise ValueError("the logits of a row are not adjacent")
    if T > 1 and logits.stride(0) < E:
        raise ValueError(f"the logits' rows overlap: they are {logits.stride(0)} apart, of {E} experts")
    return logits.stride(0) if T > 1 else E


class MoeRoute(_Moe):
    """hocf_moe_route: logits [T][E] (rows may be apart) -> experts [T][topk], weights
    [T][topk] and, with counts=True, the tokens of each expert [E]."""

    def __init__(self, T, E, topk, logits, bias=None, score=hocf.HOCF_SCORE_SOFTMAX, n_group=1, topk_group=1,
                 group_top=1, renorm=False, scale=1.0, counts=False):
        ld = _rows_ld(logits, T, E)
        _dense(torch.float32, (E,), bias=bias)
        _on(logits.device, bias=bias)
        self.logits, self.bias = logits, bias
        self.experts = torch.empty((T, topk), dtype=torch.int32, device=logits.device)
        self.weights = torch.empty((T, topk), dtype=torch.float32, device=logits.device)
        self.counts = torch.empty(E, dtype=torch.int32, device=logits.device) if counts else None
        args = (T, E, topk, torch_dt(logits), logits.data_ptr(), ld, hocf.ptr(bias), score, n_group, topk_group,
                group_top, int(renorm), scale, self.experts.data_ptr(), self.weights.data_ptr(),
                hocf.ptr(self.counts))
        self._bind("hocf_moe_route", args, logits.device, hocf.hocf_moe_route_workspace_bytes(E) if counts else 0)

    def poison(self):
        self.experts.fill_(-77)
        nan_fill(self.weights)
        if self.counts is not None:
            self.counts.fill_(-77)


class MoeRouteBwd(_Moe):
    """hocf_moe_route_bwd: logits [T][E], the chosen experts [T][topk] and the gradients
    of their weights -> dlogits [T][E]."""

    def __init__(self, T, E, topk, logits, experts, dweights, score=hocf.HOCF_SCORE_SOFTMAX, renorm=False, scale=1.0):
        ld = _rows_ld(logits, T, E)
        _dense(torch.int32, (T, topk), experts=experts)
        _dense(torch.float32, (T, topk), dweights=dweights)
        _on(logits.device, experts=experts, dweights=dweights)
        self.logits, self.experts, self.dweights = logits, experts, dweights
        self.dlogits = torch.empty((T, E), dtype=tdtype(torch_dt(logits)), device=logits.device)
        args = (T, E, topk, torch_dt(logits), logits.data_ptr(), ld, experts.data_ptr(), dweights.data_ptr(), score,
                int(renorm), scale, self.dlogits.data_ptr())
        self._bind("hocf_moe_route_bwd", args, logits.device)

    def poison(self):
        nan_fill(self.dlogits)


class MoeSlots(_Moe):
    """hocf_moe_slots: experts [T][topk] -> index [T][topk], pair [bins * cap], counts [bins]."""

    def __init__(self, T, topk, bins, per_bin, cap, experts):
        _dense(torch.int32, (T, topk), experts=experts)
        dev = experts.device
        _on(dev)
        self.experts = experts
        self.index = torch.empty((T, topk), dtype=torch.int32, device=dev)
        self.pair = torch.empty(bins * cap, dtype=torch.int32, device=dev)
        self.counts = torch.empty(bins, dtype=torch.int64, device=dev)
        args = (T, topk, bins, per_bin, cap, experts.data_ptr(), self.index.data_ptr(), self.pair.data_ptr(),
                self.counts.data_ptr())
        self._bind("hocf_moe_slots", args, dev, hocf.hocf_moe_slots_workspace_bytes(T, topk, bins))

    def poison(self):
        for t in (self.index, self.pair, self.counts):
            t.fill_(-77)


class MoeCombine(_Moe):
    """hocf_moe_combine: rows [R][N], weights [T][topk], index [T][topk] (None: pair order),
    add [T][N] (None: nothing) -> out [T][N]."""

    def __init__(self, T, topk, N, rows, weights, index=None, add=None, out_dt=BF16):
        R = rows.shape[0]
        _dense(None, (R, N), rows=rows)
        _dense(torch.float32, (T, topk), weights=weights)
        _dense(torch.int32, (T, topk), index=index)
        _dense(None, (T, N), add=add)
        _on(rows.device, weights=weights, index=index, add=add)
        if add is not None and torch_dt(add) != out_dt:
            raise TypeError(f"add is {add.dtype}, not of the output's type")
        self.rows, self.weights, self.index, self.add = rows, weights, index, add
        self.out = torch.empty((T, N), dtype=tdtype(out_dt), device=rows.device)
        args = (T, topk, N, R, torch_dt(rows), out_dt, rows.data_ptr(), weights.data_ptr(), hocf.ptr(index),
                hocf.ptr(add), self.out.data_ptr())
        self._bind("hocf_moe_combine", args, rows.device)

    def poison(self):
        nan_fill(self.out)


class MoeCombineBwd(_Moe):
    """hocf_moe_combine_bwd: rows [R][N], weights [T][topk], dout [T][N], index [T][topk] and
    its inverse pair [R] (both None: pair order) -> drows [R][N], dweights [T][topk]."""

    def __init__(self, T, topk, N, rows, weights, dout, index=None, pair=None):
        R = rows.shape[0]
        _dense(None, (R, N), rows=rows)
        _dense(torch.float32, (T, topk), weights=weights)
        _dense(None, (T, N), dout=dout)
        _dense(torch.int32, (T, topk), index=index)
        _dense(torch.int32, (R,), pair=pair)
        _on(rows.device, weights=weights, dout=dout, index=index, pair=pair)
        self.rows, self.weights, self.dout, self.index, self.pair = rows, weights, dout, index, pair
        self.drows = torch.empty((R, N), dtype=tdtype(torch_dt(rows)), device=rows.device)
        self.dweights = torch.empty((T, topk), dtype=torch.float32, device=rows.device)
        args = (T, topk, N, R, torch_dt(rows), torch_dt(dout), rows.data_ptr(), weights.data_ptr(),
                dout.data_ptr(), hocf.ptr(index), hocf.ptr(pair), self.drows.data_ptr(), self.dweights.data_ptr())
        self._bind("hocf_moe_combine_bwd", args, rows.device)

    def poison(self):
        nan_fill(self.drows)
        nan_fill(self.dweights)


def w4_layout(E, N, K, group):
    """Shapes of packed 4-bit weights and of their scales (hocf_w4_pack)."""
    nb = cdiv(N, 16)
    return (E, nb, cdiv(K, 128), 64, 4), (E, nb, cdiv(K, group), 16)


def w4_pack(codes, scales, zeros=None, group=128, stream=None):
    """hocf_w4_pack: codes [E][K][N] uint8, scales (and zeros) [E][ceil(K/group)][N] bf16 ->
    (wq, scales, zeros or None) as hocf_gemv_w4 reads them.  On another stream than the current
    one, the packing is ordered behind the current one's work, and the memory of its tensors
    is not used again before it has ended, whenever they are dropped."""
    E, K, N = codes.shape
    _dense(torch.uint8, (E, K, N), codes=codes)
    _dense(torch.bfloat16, (E, cdiv(K, group), N), scales=scales, zeros=zeros)
    _on(codes.device, scales=scales, zeros=zeros)
    words, small = w4_layout(E, N, K, group)
    wq = torch.empty(words, dtype=torch.int32, device=codes.device)
    s = torch.empty(small, dtype=torch.bfloat16, device=codes.device)
    z = None if zeros is None else torch.empty(small, dtype=torch.bfloat16, device=codes.device)
    now = torch.cuda.current_stream(codes.device)
    on = now if stream is None else stream
    if isinstance(on, int):
        on = torch.cuda.ExternalStream(on, device=codes.device)
    if on.cuda_stream != now.cuda_stream:
        on.wait_stream(now)
    hocf.check(hocf.hocf_w4_pack(E, N, K, group, codes, scales, zeros, wq, s, z, on))
    if on.cuda_stream != now.cuda_stream:
        for t in (codes, scales, zeros, wq, s, z):
            if t is not None:
                t.record_stream(on)
    return wq, s, z


class GemvW4(_Moe):
    """hocf_gemv_w4: x [R / rows_per_x][K] bf16, experts [R] (None: one matrix), packed
    weights (w4_pack) -> out [R][N]."""

    def __init__(self, R, rows_per_x, E, e0, N, K, group, x, experts, wq, scales, zeros=None, out_dt=BF16):
        words, small = w4_layout(E, N, K, group)
        _dense(torch.bfloat16, (R // rows_per_x, K), x=x)
        _dense(torch.int32, (R,), experts=experts)
        _dense(torch.int32, words, wq=wq)
        _dense(torch.bfloat16, small, scales=scales, zeros=zeros)
        _on(x.device, experts=experts, wq=wq, scales=scales, zeros=zeros)
        self.x, self.experts, self.wq, self.scales, self.zeros = x, experts, wq, scales, zeros
        self.out = torch.empty((R, N), dtype=tdtype(out_dt), device=x.device)
        args = (R, rows_per_x, E, e0, N, K, group, out_dt, x.data_ptr(), hocf.ptr(experts), wq.data_ptr(),
                scales.data_ptr(), hocf.ptr(zeros), self.out.data_ptr())
        self._bind("hocf_gemv_w4", args, x.device)

    def poison(self):
        nan_fill(self.out)


# ------------------------------------------------------------ 8-bit integers

def _rows_apart(x, T, K):
    """Row stride of x [T][K]: the numbers of a row adjacent, the rows K or more apart."""
    if tuple(x.shape) != (T, K):
        raise ValueError(f"x has shape {tuple(x.shape)}, not {(T, K)}")
    if K > 1 and x.stride(1) != 1:
        raise ValueError("the numbers of a row of x are not adjacent")
    if T > 1 and x.stride(0) < K:
        raise ValueError(f"x's rows overlap: they are {x.stride(0)} apart, of {K} numbers")
    return x.stride(0) if T > 1 else K  # (the stride of a single row says nothing)


def _bf16(dy):
    if dy.dtype not in (torch.bfloat16, torch.int16):
        raise TypeError(f"dy is {dy.dtype}, not bfloat16")


class QuantI8(_Moe):
    """hocf_quant_i8: x [T][K] (rows may be apart) -> codes [T][K] int8, scales [T] of act(x);
    with keep=True (and an activation) pre_codes and pre_scales of x itself too."""

    def __init__(self, T, K, x, act=hocf.HOCF_ACT_NONE, keep=False):
        ld, dev = _rows_apart(x, T, K), x.device
        _on(dev)
        if keep and act == hocf.HOCF_ACT_NONE:
            raise ValueError("without an activation the codes are those of x already")
        self.x = x
        self.codes = torch.empty((T, K), dtype=torch.int8, device=dev)
        self.scales = torch.empty(T, dtype=torch.float32, device=dev)
        self.pre_codes = torch.empty_like(self.codes) if keep else None
        self.pre_scales = torch.empty_like(self.scales) if keep else None
        args = (T, K, torch_dt(x), x.data_ptr(), ld, act, self.codes.data_ptr(), self.scales.data_ptr(),
                hocf.ptr(self.pre_codes), hocf.ptr(self.pre_scales))
        self._bind("hocf_quant_i8", args, dev)

    def poison(self):
        for q, s in ((self.codes, self.scales), (self.pre_codes, self.pre_scales)):
            if q is not None:
                q.fill_(-128)
                nan_fill(s)


class DequantI8(_Moe):
    """hocf_dequant_i8: codes [T][K] int8, scales [T] -> out [T][K]."""

    def __init__(self, T, K, codes, scales, out_dt=BF16):
        _dense(torch.int8, (T, K), codes=codes)
        _dense(torch.float32, (T,), scales=scales)
        _on(codes.device, scales=scales)
        self.codes, self.scales = codes, scales
        self.out = torch.empty((T, K), dtype=tdtype(out_dt), device=codes.device)
        args = (T, K, out_dt, codes.data_ptr(), scales.data_ptr(), self.out.data_ptr())
        self._bind("hocf_dequant_i8", args, codes.device)

    def poison(self):
        nan_fill(self.out)


class WeightsI8(_Moe):
    """hocf_weights_i8: w [E][K][N] -> wq [E][N][K] int8, scales [E][N]."""

    def __init__(self, E, N, K, w):
        _dense(None, (E, K, N), w=w)
        _on(w.device)
        self.w = w
        self.wq = torch.empty((E, N, K), dtype=torch.int8, device=w.device)
        self.scales = torch.empty((E, N), dtype=torch.float32, device=w.device)
        args = (E, N, K, torch_dt(w), w.data_ptr(), self.wq.data_ptr(), self.scales.data_ptr())
        self._bind("hocf_weights_i8", args, w.device, hocf.hocf_weights_i8_workspace_bytes(E, N, K))

    def poison(self):
        self.wq.fill_(-128)
        nan_fill(self.scales)


class GemmI8(_Moe):
    """hocf_gemm_i8: xq [T][K], xs [T], wq [E][N][K], ws [E][N] and the groups' offsets [E + 1]
    int64 (None: one matrix for every row) -> out [T][N].  Rows of no group keep what
    out held."""

    def __init__(self, E, T, N, K, xq, xs, wq, ws, offsets=None, out_dt=BF16):
        _dense(torch.int8, (T, K), xq=xq)
        _dense(torch.float32, (T,), xs=xs)
        _dense(torch.int8, (E, N, K), wq=wq)
        _dense(torch.float32, (E, N), ws=ws)
        _dense(torch.int64, (E + 1,), offsets=offsets)
        _on(xq.device, xs=xs, wq=wq, ws=ws, offsets=offsets)
        self.xq, self.xs, self.wq, self.ws_, self.offsets = xq, xs, wq, ws, offsets
        self.out = torch.empty((T, N), dtype=tdtype(out_dt), device=xq.device)
        args = (E, T, N, K, out_dt, xq.data_ptr(), xs.data_ptr(), wq.data_ptr(), ws.data_ptr(), hocf.ptr(offsets),
                self.out.data_ptr())
        self._bind("hocf_gemm_i8", args, xq.device)

    def poison(self):
        nan_fill(self.out)


class GemvI8(_Moe):
    """hocf_gemv_i8: xq [R / rows_per_x][K], xs [R / rows_per_x], experts [R] (None: one matrix),
    wq [E][N][K], ws [E][N] -> out [R][N]."""

    def __init__(self, R, rows_per_x, E, e0, N, K, xq, xs, experts, wq, ws, out_dt=BF16):
        _dense(torch.int8, (R // rows_per_x, K), xq=xq)
        _dense(torch.float32, (R // rows_per_x,), xs=xs)
        _dense(torch.int32, (R,), experts=experts)
        _dense(torch.int8, (E, N, K), wq=wq)
        _dense(torch.float32, (E, N), ws=ws)
        _on(xq.device, xs=xs, experts=experts, wq=wq, ws=ws)
        self.xq, self.xs, self.experts, self.wq, self.ws_ = xq, xs, experts, wq, ws
        self.out = torch.empty((R, N), dtype=tdtype(out_dt), device=xq.device)
        args = (R, rows_per_x, E, e0, N, K, out_dt, xq.data_ptr(), xs.data_ptr(), hocf.ptr(experts), wq.data_ptr(),
                ws.data_ptr(), self.out.data_ptr())
        self._bind("hocf_gemv_i8", args, xq.device)

    def poison(self):
        nan_fill(self.out)


class GemmI8Dx(_Moe):
    """hocf_gemm_i8_dx: dy [T][N] bf16, wq [E][N][K], ws [E][N], offsets as GemmI8 and, for the
    gradient of what SiLU was given, pre_codes [T][K] and pre_scales [T] -> out [T][K].  Rows
    of no group keep what out held."""

    def __init__(self, E, T, N, K, dy, wq, ws, offsets=None, pre_codes=None, pre_scales=None, out_dt=BF16):
        _dense(None, (T, N), dy=dy)
        _bf16(dy)
        _dense(torch.int8, (E, N, K), wq=wq)
        _dense(torch.float32, (E, N), ws=ws)
        _dense(torch.int64, (E + 1,), offsets=offsets)
        _dense(torch.int8, (T, K), pre_codes=pre_codes)
        _dense(torch.float32, (T,), pre_scales=pre_scales)
        _on(dy.device, wq=wq, ws=ws, offsets=offsets, pre_codes=pre_codes, pre_scales=pre_scales)
        self.dy, self.wq, self.ws_, self.offsets = dy, wq, ws, offsets
        self.pre_codes, self.pre_scales = pre_codes, pre_scales
        self.out = torch.empty((T, K), dtype=tdtype(out_dt), device=dy.device)
        args = (E, T, N, K, out_dt, dy.data_ptr(), wq.data_ptr(), ws.data_ptr(), hocf.ptr(offsets),
                hocf.ptr(pre_codes), hocf.ptr(pre_scales), self.out.data_ptr())
        self._bind("hocf_gemm_i8_dx", args, dy.device)

    def poison(self):
        nan_fill(self.out)


class GemmI8Dw(_Moe):
    """hocf_gemm_i8_dw: xq [T][K], xs [T], dy [T][N] bf16, offsets as GemmI8 -> out [E][K][N]."""

    def __init__(self, E, T, N, K, xq, xs, dy, offsets=None, out_dt=F32):
        _dense(torch.int8, (T, K), xq=xq)
        _dense(torch.float32, (T,), xs=xs)
        _dense(None, (T, N), dy=dy)
        _bf16(dy)
        _dense(torch.int64, (E + 1,), offsets=offsets)
        _on(xq.device, xs=xs, dy=dy, offsets=offsets)
        self.xq, self.xs, self.dy, self.offsets = xq, xs, dy, offsets
        self.out = torch.empty((E, K, N), dtype=tdtype(out_dt), device=xq.device)
        args = (E, T, N, K, out_dt, xq.data_ptr(), xs.data_ptr(), dy.data_ptr(), hocf.ptr(offsets), self.out.data_ptr())
        self._bind("hocf_gemm_i8_dw", args, xq.device, hocf.hocf_gemm_i8_dw_workspace_bytes(E, T, N, K))

    def poison(self):
        nan_fill(self.out)
