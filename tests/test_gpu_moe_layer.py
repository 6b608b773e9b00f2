"""The mixture-of-experts operators together: the layer and the decode step of
computation_collective_amd/moe_layer.py against plain 64-bit implementations,
stage by stage, and the operators on streams, in graphs and far into large
buffers."""

import numpy as np
import pytest
import torch

import moe_ref as ref
from computation_collective_amd import buffers as bf
from computation_collective_amd import hocf
from computation_collective_amd import moe_layer
from test_gpu_moe import dev, host, near, run, say, w4_case, w4_steps

pytestmark = pytest.mark.gpu
SOFTMAX, SIGMOID = hocf.HOCF_SCORE_SOFTMAX, hocf.HOCF_SCORE_SIGMOID


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


def normal(shape, seed, std=1.0):
    return (std * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).bfloat16().cuda()


def silu(y):
    return y / (1 + np.exp(-y))


@pytest.mark.parametrize("P,E,B,topk,score,renorm", [(1, 4, 20, 2, SOFTMAX, True), (2, 2, 24, 2, SOFTMAX, False),
                                                     (4, 3, 70, 4, SIGMOID, True)])
def test_layer(P, E, B, topk, score, renorm):
    say(f"layer P={P} E={E} B={B} topk={topk} score={score}")
    K, H, n = 256, 256, P * E
    w_up, w_down = normal((n, K, H), 1, 0.06), normal((n, H, K), 2, 0.06)
    layer = moe_layer.MoeLayer(P, E, B, topk, normal((K, n), 3, 0.06), w_up, w_down, cap=B * topk,
                               recv_rows=P * B * topk + E * 256, score=score, renorm=renorm)
    x, dout = normal((P, B, K), 4), normal((P, B, K), 5)
    for again in range(2):
        layer.windows.fill_(float("nan"))
        out = layer.forward(x)
        drows, dlogits = layer.backward(dout)
        torch.cuda.synchronize()
    logits = host(layer.logits)
    e, w, c = ref.route(logits, topk, score=score, renorm=renorm)
    assert np.array_equal(layer.route.experts.cpu().numpy(), e)
    assert np.array_equal(layer.route.counts.cpu().numpy(), c)
    near(layer.route.weights, w, np.abs(w), torch.float32, 40)
    weights = layer.route.weights.cpu().numpy().reshape(P, B, topk)
    xs, up, down = host(x), host(w_up), host(w_down)
    for s in range(P):
        index, pair, _ = ref.slots(e.reshape(P, B, topk)[s], P, E, layer.cap)
        assert np.array_equal(layer.slots[s].index.cpu().numpy(), index)
        rows = host(layer.windows[s].reshape(-1, K))
        for t in range(B):
            for j in range(topk):
                k = e.reshape(P, B, topk)[s, t, j]
                # roundings: y and silu(y) to bf16 (half steps of 2^-8, the slope of silu is below 1.1) and the
                # row; K + H products in fp32
                y = xs[s, t] @ up[k]
                ey = 2.0 ** -8 * np.abs(y) + ref.rel_steps(2 * K) * (np.abs(xs[s, t]) @ np.abs(up[k]))
                h = silu(y)
                eh = 1.1 * ey + 2.0 ** -8 * (np.abs(h) + 1.1 * ey) + ref.rel_steps(8) * np.abs(h)
                want = h @ down[k]
                room = eh @ np.abs(down[k]) * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want) + \
                    ref.rel_steps(2 * H) * ((np.abs(h) + eh) @ np.abs(down[k]))
                got = rows[index[t, j]]
                assert not np.isnan(got).any() and (np.abs(got - want) <= room).all()
        want, size = ref.combine(rows, weights[s], index, xs[s])
        near(out[s], want, size, torch.bfloat16, topk + 1)
        dr, dw, size = ref.combine_bwd(rows, weights[s], host(dout)[s], index)
        near(drows[s], dr, np.abs(dr), torch.bfloat16, 1)
        near(layer.dweights.view(P, B, topk)[s], dw, size, torch.float32, K / 64 + 10)
    d, size = ref.route_bwd(logits, e, layer.dweights.cpu().numpy(), score, renorm, 1.0)
    near(dlogits, d, size, torch.bfloat16, 80)


def test_layer_refuses_what_its_windows_do_not_hold():
    K, H = 256, 256
    layer = moe_layer.MoeLayer(1, 2, 8, 2, normal((K, 2), 3), normal((2, K, H), 1), normal((2, H, K), 2), cap=15,
                               recv_rows=1024)
    with pytest.raises(RuntimeError, match="its window holds 15"):
        layer.forward(normal((1, 8, K), 4))
    layer = moe_layer.MoeLayer(1, 2, 8, 2, normal((K, 2), 3), normal((2, K, H), 1), normal((2, H, K), 2), cap=16,
                               recv_rows=256)
    with pytest.raises(RuntimeError, match="rank 0"):
        layer.forward(normal((1, 8, K), 4))


def decode_of(T, E, topk, K, H, group):
    up, down = w4_case(E, H, K, group, True, 1), w4_case(E, K, H, group, False, 2)
    d = moe_layer.MoeDecode(T, E, topk, normal((K, E), 3, 0.06), bf.w4_pack(*[a.cuda() for a in up], group),
                            bf.w4_pack(down[0].cuda(), down[1].cuda(), None, group), K, H, group)
    return d, up, down


def check_decode(d, T, E, topk, K, H, group, up, down, x, out):
    e, w, _ = ref.route(host(d.logits), topk, renorm=True)
    assert np.array_equal(d.route.experts.cpu().numpy(), e)
    y, size = ref.w4(host(x), up[0].numpy(), up[1].float().numpy(), up[2].float().numpy(), e.reshape(-1), 0, topk, group)
    got = host(d.hidden)
    ey = 2.0 ** -8 * np.abs(y) + ref.rel_steps(w4_steps(K, group)) * size
    assert (np.abs(got - silu(y)) <= 1.1 * ey + 2.0 ** -8 * (np.abs(silu(y)) + 1.1 * ey) + 2.0 ** -20).all()
    y, size = ref.w4(got, down[0].numpy(), down[1].float().numpy(), None, e.reshape(-1), 0, 1, group)
    near(d.down.out, y, size, torch.bfloat16, w4_steps(H, group))
    want, size = ref.combine(host(d.down.out), d.route.weights.cpu().numpy(), None, host(x))
    near(out, want, size, torch.bfloat16, topk + 1)


@pytest.mark.parametrize("T,E,topk,K,H,group", [(1, 8, 2, 256, 136, 32), (4, 4, 3, 264, 512, 128), (9, 16, 1, 128, 64, 64)])
def test_decode(T, E, topk, K, H, group):
    say(f"decode T={T} E={E} topk={topk} {K} -> {H} group={group}")
    d, up, down = decode_of(T, E, topk, K, H, group)
    for seed in (7, 8):
        x = normal((T, K), seed)
        out = d.step(x)
        torch.cuda.synchronize()
        check_decode(d, T, E, topk, K, H, group, up, down, x, out)


def test_decode_in_a_graph():
    """Captured once, replayed on new inputs, with eager work and waits between the replays."""
    T, E, topk, K, H, group = 3, 8, 2, 256, 136, 64
    say("decode in a graph")
    d, up, down = decode_of(T, E, topk, K, H, group)
    eager, _, _ = decode_of(T, E, topk, K, H, group)
    d.step(normal((T, K), 1))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d.experts()
    for seed in range(4):
        x = normal((T, K), 10 + seed)
        want = eager.step(x).clone()
        d.x.copy_(x)
        d.logits.copy_(eager.logits)
        graph.replay()
        if seed % 2:
            torch.cuda.synchronize()
        assert torch.equal(d.combine.out.view(torch.bfloat16), want)


def test_training_operators_in_a_graph():
    """Router with counts, window rows, weighted sum and both gradients: every replay equals the eager calls."""
    T, E, topk, N, bins = 1500, 40, 4, 264, 5
    say("training operators in a graph")
    cap = T * topk // bins + 900

    def build():
        h = {}
        h["logits"] = torch.zeros((T, E), device="cuda")
        h["rows"] = torch.zeros((bins * cap, N), dtype=torch.bfloat16, device="cuda")
        h["dout"] = torch.zeros((T, N), device="cuda")
        h["route"] = bf.MoeRoute(T, E, topk, h["logits"], score=SIGMOID, renorm=True, counts=True)
        h["slots"] = bf.MoeSlots(T, topk, bins, E // bins, cap, h["route"].experts)
        h["combine"] = bf.MoeCombine(T, topk, N, h["rows"], h["route"].weights, index=h["slots"].index)
        h["cbwd"] = bf.MoeCombineBwd(T, topk, N, h["rows"], h["route"].weights, h["dout"], index=h["slots"].index,
                                     pair=h["slots"].pair)
        h["rbwd"] = bf.MoeRouteBwd(T, E, topk, h["logits"], h["route"].experts, h["cbwd"].dweights, score=SIGMOID,
                                   renorm=True)
        return h

    def call(h):
        for k in ("route", "slots", "combine", "cbwd", "rbwd"):
            h[k].run()

    def fill(h, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        h["logits"].copy_(torch.randn(T, E, generator=g, device="cuda"))
        h["rows"].copy_(torch.randn(bins * cap, N, generator=g, device="cuda"))
        h["dout"].copy_(torch.randn(T, N, generator=g, device="cuda"))

    def outputs(h):
        return [h["route"].experts, h["route"].weights, h["route"].counts, h["slots"].index, h["slots"].pair,
                h["slots"].counts, h["combine"].out, h["cbwd"].drows, h["cbwd"].dweights, h["rbwd"].dlogits]

    a, b = build(), build()
    fill(a, 0)
    call(a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(a)
    for seed in range(1, 5):
        fill(a, seed)
        fill(b, seed)
        call(b)
        graph.replay()
        if seed % 2:
            torch.cuda.synchronize()
        for i, (x, y) in enumerate(zip(outputs(a), outputs(b))):
            assert torch.equal(x, y), (seed, i)
        assert not a["route"].ws.any()


def test_on_another_stream():
    """The current stream's, and one that is given: behind work of that stream."""
    T, E, topk = 5000, 64, 4
    say("on another stream")
    x = torch.zeros((T, E), device="cuda")
    want = torch.randn((T, E), generator=torch.Generator().manual_seed(1)).cuda()
    eager = run(bf.MoeRoute(T, E, topk, want, counts=True))
    h = bf.MoeRoute(T, E, topk, x, counts=True)
    torch.cuda.synchronize()
    side, busy = torch.cuda.Stream(), torch.randn(2048, 2048, device="cuda")
    for given in (False, True):
        x.zero_()
        h.poison()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(8):
                busy = busy @ busy * 1e-3                  # (the logits are written only after these)
            x.copy_(want)
            if not given:
                h.run()
        if given:
            h.run(side)
        side.synchronize()
        assert torch.equal(h.experts, eager.experts) and torch.equal(h.weights, eager.weights)
        assert torch.equal(h.counts, eager.counts)


# ------------------------------------------------------------------ far into large buffers

def test_route_far_rows():
    """Logits rows 2^24 apart: the last rows begin beyond 2^31 elements and 2^32 bytes."""
    T, E, topk, ld = 140, 60, 4, 1 << 24
    say("route far rows")
    store = torch.empty((T, ld), dtype=torch.bfloat16, device="cuda")
    x = store[:, :E]
    x.copy_(torch.randn((T, E), generator=torch.Generator().manual_seed(2)))
    h = run(bf.MoeRoute(T, E, topk, x, renorm=True))
    near_ = run(bf.MoeRoute(T, E, topk, x.contiguous(), renorm=True))
    assert torch.equal(h.experts, near_.experts) and torch.equal(h.weights, near_.weights)
    dw = torch.randn((T, topk), generator=torch.Generator().manual_seed(3)).cuda()
    a = run(bf.MoeRouteBwd(T, E, topk, x, h.experts, dw))
    b = run(bf.MoeRouteBwd(T, E, topk, x.contiguous(), h.experts, dw))
    assert torch.equal(a.dlogits, b.dlogits)


def test_combine_far_rows():
    """Rows beyond 2^31 elements; a row's gradient and the zeros around it land there too."""
    R, N, T, topk = 270000, 8192, 6, 2
    say("combine far rows")
    assert (R - 12) * N > 2 ** 31
    rows = torch.empty((R, N), dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([R - 1, 0, R - 2, 1, R - 12, R // 2, 7, R - 3, -1, 262144, 262143, -1])
    index = at.view(T, topk).int().cuda()
    pair = torch.full((R,), -1, dtype=torch.int32)
    pair[at[at >= 0]] = torch.arange(T * topk, dtype=torch.int32)[at >= 0]
    few = normal((T * topk, N), 1)
    rows[at[at >= 0].cuda()] = few[(at >= 0).cuda()]
    w, dout = torch.rand((T, topk), generator=torch.Generator().manual_seed(2)).cuda(), normal((T, N), 3)
    out = run(bf.MoeCombine(T, topk, N, rows, w, index=index)).out
    inner = torch.arange(T * topk).masked_fill(at < 0, -1).view(T, topk).int().cuda()
    want = run(bf.MoeCombine(T, topk, N, few, w, index=inner)).out
    assert torch.equal(out, want)
    b = run(bf.MoeCombineBwd(T, topk, N, rows, w, dout, index=index, pair=pair.cuda()))
    s = run(bf.MoeCombineBwd(T, topk, N, few, w, dout, index=inner, pair=inner.view(-1)))
    assert torch.equal(b.dweights, s.dweights)
    keep = (at >= 0).cuda()
    assert torch.equal(b.drows[at[at >= 0].cuda()], s.drows[keep])
    b.drows[at[at >= 0].cuda()] = 0
    assert not b.drows.any()


def test_w4_far_experts():
    """Packed weights beyond 2^32 bytes."""
    E, N, K, group = 520, 4096, 4096, 128
    say("w4 far experts")
    words, small = bf.w4_layout(E, N, K, group)
    wq = torch.empty(words, dtype=torch.int32, device="cuda")
    scales = torch.empty(small, dtype=torch.bfloat16, device="cuda")
    assert wq.numel() * 4 > 2 ** 32
    g = torch.Generator(device="cuda").manual_seed(1)
    for e in (0, 1, E - 1):
        wq[e] = torch.randint(-2 ** 31, 2 ** 31, words[1:], generator=g, device="cuda").int()
        scales[e] = 0.01 * torch.rand(small[1:], generator=g, device="cuda") + 0.01
    x = normal((2, K), 2)
    h = run(bf.GemvW4(2, 1, E, 0, N, K, group, x, dev(np.array([E - 1, 1], np.int32)), wq, scales))
    for r, e in enumerate((E - 1, 1)):
        one = run(bf.GemvW4(1, 1, 1, 0, N, K, group, x[r:r + 1], None, wq[e:e + 1], scales[e:e + 1]))
        near(h.out[r], host(one.out)[0], np.abs(host(one.out)[0]), torch.bfloat16, 0)
