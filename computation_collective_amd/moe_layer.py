"""A mixture-of-experts layer from the library's operators.

Two forms, both on one GPU:

* ``MoeLayer``, for training and prompts: P logical ranks of B tokens, E experts
  each.  route -> dispatch + up projection (hocf_a2a_gemm) -> SiLU -> down
  projection + combine windows (hocf_gemm_a2a) -> the windows' rows of each pair
  (hocf_moe_slots) -> the tokens' weighted sums plus the residual
  (hocf_moe_combine); and, from the gradient of the outputs, the gradients of
  the experts' rows, the weights (hocf_moe_combine_bwd) and the router's logits
  (hocf_moe_route_bwd).
* ``MoeDecode``, for a decode step of a few tokens: route -> up and down
  projections with 4-bit weights (hocf_gemv_w4) -> weighted sum.

Buffers are allocated once; a step launches on the current stream.  The library
is called through its Python binding; matrix products with the router and the
activation are plain torch operations.

    python -m computation_collective_amd.moe_layer

runs both at the sizes of the dispatch and combine workloads and prints the
time of a step.
"""

from __future__ import annotations

import argparse

import torch

from . import buffers as bf
from . import configs as cfgs
from . import hocf


def silu_(x: torch.Tensor) -> torch.Tensor:
    return torch.nn.functional.silu(x, inplace=True)


class MoeLayer:
    """w_router [K][P*E] bf16, w_up [P*E][K][H] and w_down [P*E][H][K] bf16.

    forward(X [P][B][K] bf16) -> out [P][B][K] bf16 (the residual X included);
    backward(dout) -> (drows [P][P*cap][K], dlogits [P*B][P*E]): the gradients
    that the experts' and the router's own products take (those products, and
    the way of drows back to the experts' ranks, are not part of the layer).
    `cap`: rows one rank sends to one source at most.  `recv_rows`: rows one rank
    receives at most (its experts' groups padded to 256).  forward() raises where
    a batch needs more of either, and computes the next one that does not.  B *
    topk is a multiple of 4 (every rank's choices start on 16 bytes).

    The operators' error words are read where forward() waits for the device
    anyway, and by check(), which waits: an error of the last operators of a step
    is raised by the next forward(), or by a check() after the step."""

    def __init__(self, P, E, B, topk, w_router, w_up, w_down, cap, recv_rows, score=hocf.HOCF_SCORE_SOFTMAX,
                 renorm=True):
        self.P, self.E, self.B, self.topk, self.cap = P, E, B, topk, cap
        self.K, self.H = w_up.shape[1], w_up.shape[2]
        self.w_router = w_router
        self.X = torch.empty((P, B, self.K), dtype=torch.bfloat16, device=w_up.device)
        self.logits = torch.empty((P * B, P * E), dtype=torch.bfloat16, device=w_up.device)
        self.dout = torch.empty_like(self.X)
        how = dict(score=score, renorm=renorm)
        self.route = bf.MoeRoute(P * B, P * E, topk, self.logits, counts=True, **how)
        experts = self.route.experts.view(P, B, topk)
        weights = self.route.weights.view(P, B, topk)
        self.dispatch = [bf.A2aGemm(P, E, p * E, B, topk, self.H, self.K, bf.BF16, self.X, experts,
                                    w_up[p * E:(p + 1) * E], recv_rows, device=w_up.device) for p in range(P)]
        self.w_down = w_down
        # windows[s][p]: what rank p sends back to source s; one source's windows follow one another
        self.windows = torch.empty((P, P, cap, self.K), dtype=torch.bfloat16, device=w_up.device)
        self.flags = torch.zeros((P, P, 4), dtype=torch.int32, device=w_up.device)
        self.win = [hocf.windows([(self.windows[s, p], self.flags[s, p]) for s in range(P)]) for p in range(P)]
        ws = hocf.hocf_gemm_a2a_workspace_bytes(P)
        self.ws = torch.zeros((ws + 3) // 4 + 4, dtype=torch.int32, device=w_up.device)
        self.epoch = 0
        self.slots = [bf.MoeSlots(B, topk, P, E, cap, experts[s]) for s in range(P)]
        rows = [self.windows[s].view(P * cap, self.K) for s in range(P)]
        self.combine = [bf.MoeCombine(B, topk, self.K, rows[s], weights[s], index=self.slots[s].index, add=self.X[s])
                        for s in range(P)]
        self.combine_bwd = [bf.MoeCombineBwd(B, topk, self.K, rows[s], weights[s], self.dout[s],
                                             index=self.slots[s].index, pair=self.slots[s].pair) for s in range(P)]
        self.dweights = torch.empty((P * B, topk), dtype=torch.float32, device=w_up.device)
        self.route_bwd = bf.MoeRouteBwd(P * B, P * E, topk, self.logits, self.route.experts, self.dweights, **how)
        # one error word for every operator that can report one
        parts = [(f"rank {p}: dispatch", self.dispatch[p]) for p in range(P)]
        parts += [(f"source {s}: weighted sum", self.combine[s]) for s in range(P)]
        parts += [(f"source {s}: backward pass of the weighted sum", self.combine_bwd[s]) for s in range(P)]
        parts += [("backward pass of the router", self.route_bwd)]
        self.status = torch.zeros(len(parts) + P, dtype=torch.int32, device=w_up.device)
        for i, (_, handle) in enumerate(parts):
            handle.report_to(self.status[i:i + 1])
        self.reporters = [name for name, _ in parts] + [f"rank {p}: down projection" for p in range(P)]

    def check(self):
        """Raises what an operator has reported since the last check; waits for the stream."""
        words = self.status.tolist()
        if any(words):
            self.status.zero_()
            raise RuntimeError("; ".join(f"{name}: {hocf.status_string(w)}"
                                         for name, w in zip(self.reporters, words) if w))

    def forward(self, X):
        P, E = self.P, self.E
        self.X.copy_(X)
        torch.mm(self.X.view(P * self.B, self.K), self.w_router, out=self.logits)
        self.route.run()
        for s in range(P):
            self.slots[s].run()
        for p in range(P):
            self.dispatch[p].run()
        # the down projection takes its layout from the host
        for p in range(P):
            d = self.dispatch[p]
            offsets, sent = d.offsets.cpu().numpy(), d.send_counts.cpu().numpy()
            self.check()
            if sent.max() > self.cap:
                raise RuntimeError(f"rank {p} sends {sent.max()} rows to one source, its window holds {self.cap}")
            y = d.Y.view(torch.bfloat16)
            silu_(y[:int(offsets[-1])])
            self.epoch = self.epoch % 0xFFFFFFF0 + 1
            hocf.check(hocf.hocf_gemm_a2a(
                P, E, int(offsets[-1]), self.K, self.H, bf.BF16, bf.BF16, d.Y, self.w_down[p * E:(p + 1) * E], offsets,
                d.dest, d.slot, sent, self.win[p], self.cap, 256, 256,
                hocf.sync(self.epoch, self.ws, self.ws.numel() * 4 - 16, status=self.status[p - P:].data_ptr()),
                torch.cuda.current_stream(self.X.device)))
        for s in range(P):
            self.combine[s].run()
        return torch.stack([c.out.view(torch.bfloat16) for c in self.combine])

    def backward(self, dout):
        P = self.P
        self.dout.copy_(dout)
        for s in range(P):
            self.combine_bwd[s].run()
            self.dweights[s * self.B:(s + 1) * self.B].copy_(self.combine_bwd[s].dweights)
        self.route_bwd.run()
        return (torch.stack([c.drows.view(torch.bfloat16) for c in self.combine_bwd]),
                self.route_bwd.dlogits.view(torch.bfloat16))


class MoeDecode:
    """A decode step of T tokens over E experts with 4-bit weights: `up` (K -> H) and
    `down` (H -> K) as bf.w4_pack gives them, w_router [K][E] bf16.  step(x [T][K]
    bf16) -> [T][K] bf16, the residual x included."""

    def __init__(self, T, E, topk, w_router, up, down, K, H, group, score=hocf.HOCF_SCORE_SOFTMAX, renorm=True):
        dev = w_router.device
        self.w_router = w_router
        self.x = torch.empty((T, K), dtype=torch.bfloat16, device=dev)
        self.logits = torch.empty((T, E), dtype=torch.bfloat16, device=dev)
        self.route = bf.MoeRoute(T, E, topk, self.logits, score=score, renorm=renorm)
        experts = self.route.experts.view(-1)
        self.up = bf.GemvW4(T * topk, topk, E, 0, H, K, group, self.x, experts, *up)
        self.hidden = self.up.out.view(torch.bfloat16)
        self.down = bf.GemvW4(T * topk, 1, E, 0, K, H, group, self.hidden, experts, *down)
        self.combine = bf.MoeCombine(T, topk, K, self.down.out, self.route.weights, add=self.x)

    def step(self, x):
        self.x.copy_(x)
        torch.mm(self.x, self.w_router, out=self.logits)
        return self.experts()

    def experts(self):
        """What follows the router's logits (self.logits, self.x): can be captured into a graph."""
        self.route.run()
        self.up.run()
        silu_(self.hidden)
        self.down.run()
        self.combine.run()
        return self.combine.out.view(torch.bfloat16)


def _timed(fn, steps):
    for _ in range(3):
        fn()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(steps):
        fn()
    end.record()
    end.synchronize()
    return start.elapsed_time(end) / steps


def random_w4(E, K, N, group, gen, device):
    codes = torch.randint(0, 16, (E, K, N), generator=gen, dtype=torch.uint8, device=device)
    scales = (0.002 * (0.5 + torch.rand(E, -(-K // group), N, generator=gen, device=device))).bfloat16()
    return bf.w4_pack(codes, scales, None, group)


def main(argv=None):
    c = cfgs.A2A_GEMM_MOE
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--ranks", type=int, default=c.P)
    ap.add_argument("--tokens", type=int, default=c.B, help="tokens of one rank")
    ap.add_argument("--decode-tokens", type=int, default=4)
    ap.add_argument("--steps", type=int, default=10)
    a = ap.parse_args(argv)
    P, E, B, topk, K, H = a.ranks, c.E, a.tokens, c.topk, c.K, c.N
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev).manual_seed(0)

    def normal(*shape, std=1.0):
        return (std * torch.randn(shape, generator=gen, device=dev)).bfloat16()

    pairs = B * topk // P                  # of one source on one rank, on average
    layer = MoeLayer(P, E, B, topk, normal(K, P * E, std=K ** -0.5), normal(P * E, K, H, std=0.02),
                     normal(P * E, H, K, std=0.02), cap=2 * pairs + 64, recv_rows=2 * P * pairs + E * 256)
    X, dout = normal(P, B, K), normal(P, B, K)
    layer.backward(layer.forward(X))
    layer.check()
    print(f"layer, {P} ranks x {B} tokens, top-{topk} of {P * E} experts {K} -> {H} -> {K}: "
          f"forward {_timed(lambda: layer.forward(X), a.steps):.3f} ms, "
          f"backward of combine and router {_timed(lambda: layer.backward(dout), a.steps):.3f} ms")
    T, E, group = a.decode_tokens, P * E, 128
    decode = MoeDecode(T, E, topk, normal(K, E, std=K ** -0.5), random_w4(E, K, H, group, gen, dev),
                       random_w4(E, H, K, group, gen, dev), K, H, group)
    x = normal(T, K)
    print(f"decode, {T} tokens, top-{topk} of {E} experts, 4-bit weights: "
          f"step {1e3 * _timed(lambda: decode.step(x), 20 * a.steps):.1f} us")


if __name__ == "__main__":
    main()
