"""The 8-bit layer as a user runs it: norm, router, plan, prefetch of 8-bit weight
rows, 8-bit dispatch, gate and up, down, combine, and the router's backward from
combine's.  Every step against 64 bits on the values the step before left, then
the whole chain captured into a graph, and two chains at once on two streams."""
import numpy as np
import pytest
import torch

import load_balancing_amd as mx
from gpu_harness import bf16_dev, bits, to_dev
from quant_ref import check_rows, host, scale_bytes, values, weight_values

pytestmark = pytest.mark.gpu


def f64(t):
    return t.double().cpu().numpy()


class Layer:
    """Static buffers of one layer and its forward (and the router's backward)."""

    def __init__(self, R=4, E=16, S=37, K=4, H=272, F=208, B=2, seed=0, score=mx.SCORE_SIGMOID, groups=4):
        dev = "cuda"
        self.s = s = mx.Shape(R, E, S, K, H)
        self.F, self.B = F, B
        self.opts = mx.RouterOpts(score, True, groups, mx.F32, 2.0)
        self.b = mx.allocate(mx.Shape(R, E, S, K, 8))
        rng = np.random.default_rng(seed)
        self.rng = rng
        e = lambda shape, t: torch.empty(shape, dtype=t, device=dev)  # noqa: E731
        N, NK = s.N, s.NK
        f32, i32, bf, u8 = torch.float32, torch.int32, torch.bfloat16, torch.uint8
        self.x, self.res, self.res_out, self.y16 = (e((N, H), bf) for _ in range(4))
        self.norm_w = torch.ones(H, dtype=bf, device=dev)
        self.y8, self.ys = e((N, H), torch.float8_e4m3fn), e((N, scale_bytes(H)), torch.float8_e8m0fnu)
        self.w_router = to_dev(rng.standard_normal((H, E)).astype(np.float32) * H ** -0.5)
        self.logits = e((N, E), f32)
        self.topk, self.gates = e(NK, i32), e(NK, f32)
        self.counts, self.prob, self.loss = e((groups, E), i32), e((groups, E), f32), e(1, f32)
        self.ws = e(mx.moonep_router_workspace_bytes(s, self.opts), u8)
        # weights: bf16 rows of gate, up and down, and their 8-bit rows
        mats = [(F, H), (F, H), (H, F)]
        n = [o * i for o, i in mats]
        self.w16 = bf16_dev(self.bf(rng.standard_normal((E, sum(n))) * 0.1))
        at, self.win = 0, []
        for o, i in mats:
            code, at = at, at + o * i
            scale, at = at, at + -(-o // 128) * scale_bytes(i)
            at += -at % 16
            self.win.append((code, scale))
        self.stride = at
        self.w8 = torch.zeros((E, at), dtype=u8, device=dev)
        off = 0
        for (o, i), (code, scale), m in zip(mats, self.win, n):
            mx.moonep_quant_weights(s, i, o, self.w16, sum(n), off, self.w8, at, code, scale)
            off += m
        self.mats, self.pool = mats, torch.zeros((R * B, at), dtype=u8, device=dev)
        self.wslot = e(E + R, i32)
        self.buf8, self.bufs = e((NK, H), torch.float8_e4m3fn), e((NK, scale_bytes(H)), u8)
        self.h8, self.hs = e((NK, F), torch.float8_e4m3fn), e((NK, scale_bytes(F)), u8)
        self.out, self.y = e((NK, H), bf), e((N, H), bf)
        self.dy, self.d_out, self.d_gates = e((N, H), bf), e((NK, H), bf), e(NK, f32)
        self.d_loss = torch.full((1,), 0.01, device=dev)
        self.d_logits = e((N, E), f32)

    @staticmethod
    def bf(v):
        return torch.from_numpy(np.ascontiguousarray(v, dtype=np.float32)).bfloat16().view(torch.int16).numpy().view(np.uint16)

    def load(self, seed):
        rng = np.random.default_rng(1000 + seed)
        shape = (self.s.N, self.s.H)
        for t, scale in ((self.x, 1.0), (self.res, 3.0), (self.dy, 1.0)):
            t.copy_(bf16_dev(self.bf(rng.standard_normal(shape) * scale)).view(shape))
        for t in self.outputs().values():
            t.view(torch.uint8).fill_(0x5B)

    def forward(self):
        s, b, H, F, B = self.s, self.b, self.s.H, self.F, self.B
        mx.moonep_rmsnorm_quant(s, self.x, self.res, self.norm_w, 1e-6, self.res_out, self.y16, self.y8, self.ys)
        torch.matmul(self.y16.float(), self.w_router, out=self.logits)
        mx.moonep_router(s, self.opts, self.logits, self.topk, self.gates, self.counts, self.prob, self.loss, self.ws)
        mx.moonep_route_stats(s, self.topk, b.expert_counts, b.maxvio, b.workspace)
        mx.moonep_plan(s, self.topk, b.expert_counts, b.workspace, b.plan, b.slot_of, b.src_of_slot)
        mx.moonep_weight_slots(s, b.plan, B, self.wslot)
        mx.moonep_prefetch_weights(s, b.plan, self.wslot, B, self.stride, self.w8, self.pool)
        mx.moonep_dispatch_quant(s, self.y8, self.ys, b.slot_of, self.buf8, self.bufs)
        mx.moonep_expert_glu_quant(s, b.plan, self.wslot, B, H, F, self.buf8, self.bufs, self.w8, self.pool, self.stride,
                                   *self.win[0], *self.win[1], self.h8, self.hs)
        mx.moonep_expert_gemm_quant(s, b.plan, self.wslot, B, F, H, self.h8, self.hs, self.w8, self.pool, self.stride,
                                    *self.win[2], self.out)
        mx.moonep_combine(s, self.out, self.gates, b.slot_of, self.y)

    def backward(self):
        mx.moonep_combine_bwd(self.s, self.dy, self.out, self.gates, self.b.slot_of, self.d_out, self.d_gates)
        mx.moonep_router_bwd(self.s, self.opts, self.logits, self.topk, self.counts, self.d_gates, self.d_loss,
                             self.d_logits)

    def outputs(self):
        return dict(res_out=self.res_out, y16=self.y16, y8=self.y8, ys=self.ys, logits=self.logits, topk=self.topk,
                    gates=self.gates, counts=self.counts, prob=self.prob, loss=self.loss, slot_of=self.b.slot_of,
                    buf8=self.buf8, bufs=self.bufs, h8=self.h8, hs=self.hs, out=self.out, y=self.y, d_out=self.d_out,
                    d_gates=self.d_gates, d_logits=self.d_logits, wslot=self.wslot, ws=self.ws, pool=self.pool)

    def snapshot(self):
        skip = ("ws", "pool")  # scratch, and slots that no replica of this plan has
        return {k: v.view(torch.uint8).cpu().numpy().copy() for k, v in self.outputs().items() if k not in skip}


def test_chain_step_by_step():
    L = Layer()
    L.load(0)
    L.forward()
    L.backward()
    torch.cuda.synchronize()
    s, b, N, K, E, H, F = L.s, L.b, L.s.N, L.s.K, L.s.E, L.s.H, L.F
    assert mx.moonep_read_error(b.workspace) == 0
    r = f64(L.res_out)
    want = r / np.sqrt((r * r).mean(1, keepdims=True) + 1e-6)
    check_rows(host(L.y8), host(L.ys), want, np.abs(want) * (H + 8) * 2.0 ** -24)
    # ids and gates of the logits as they are; counts as the plan's statistics
    l = f64(L.logits)
    ids = np.argsort(-l, axis=1, kind="stable")[:, :K]
    np.testing.assert_array_equal(L.topk.cpu().numpy().reshape(N, K), ids)
    sc = np.take_along_axis(1 / (1 + np.exp(-l)), ids, 1)
    np.testing.assert_allclose(L.gates.cpu().numpy().reshape(N, K), 2 * sc / sc.sum(1, keepdims=True),
                               rtol=(4 * np.abs(l).max() + 40) * 2.0 ** -24)
    np.testing.assert_allclose(f64(L.gates).reshape(N, K).sum(1), 2.0, rtol=2.0 ** -20)
    np.testing.assert_array_equal(L.counts.cpu().numpy().sum(0), b.expert_counts.cpu().numpy())
    # dispatch
    slot = b.slot_of.cpu().numpy()
    tok = np.arange(s.NK) // K
    np.testing.assert_array_equal(host(L.buf8)[slot], host(L.y8)[tok])
    np.testing.assert_array_equal(host(L.bufs)[slot], host(L.ys)[tok])
    # products: the expert of the entry at each row, from the weight rows
    expert = np.empty(s.NK, np.int64)
    expert[slot] = L.topk.cpu().numpy()
    w8 = host(L.w8)

    def product(x8, xs, which, cols):
        o, i = L.mats[which]
        code, scale = L.win[which]
        y, a = np.zeros((s.NK, o)), np.zeros((s.NK, o))
        xv = values(x8, xs)
        for e in range(E):
            wv = weight_values(w8[e, code:code + o * i].reshape(o, i),
                               w8[e, scale:scale + -(-o // 128) * scale_bytes(i)].reshape(-1, scale_bytes(i)))
            at = expert == e
            y[at], a[at] = xv[at] @ wv.T, np.abs(xv[at]) @ np.abs(wv).T
        return y, a

    (g, ga), (u, ua) = (product(host(L.buf8), host(L.bufs), m, H) for m in (0, 1))
    silu = g / (1 + np.exp(-g))
    dg, du = H * 2.0 ** -23 * ga, H * 2.0 ** -23 * ua
    h = silu * u
    check_rows(host(L.h8), host(L.hs), h,
               1.1 * dg * np.abs(u) + (np.abs(silu) + 1.1 * dg) * du + np.abs(h) * (np.abs(g) + 4) * 2.0 ** -22)
    o, oa = product(host(L.h8), host(L.hs), 2, F)
    off = np.abs(f64(L.out) - o)
    assert (off <= np.abs(o) * 2.0 ** -8 + 2 * F * 2.0 ** -23 * oa + 2.0 ** -134).all()
    # combine, one rounding of the fp64 sum
    y = (f64(L.out)[slot].reshape(N, K, H) * f64(L.gates).reshape(N, K, 1)).sum(1)
    assert (np.abs(f64(L.y) - y) <= np.abs(y) * 2.0 ** -8 + 2.0 ** -134).all()
    # and against the layer without its 8-bit roundings: a code is at most 2^-4 off
    # relative to its value (or 2^-10 of the block's scale, 448 at most), in x, in
    # the weights and in h; to first order the products add them up
    w16 = f64(L.w16.view(torch.bfloat16)).reshape(E, -1)
    n = F * H
    ref = np.zeros((N, H))
    mag = np.zeros((N, H))
    for e in range(E):
        wg, wu, wd = w16[e, :n].reshape(F, H), w16[e, n:2 * n].reshape(F, H), w16[e, 2 * n:].reshape(H, F)
        t, k = np.nonzero(ids == e)
        if not t.size:
            continue
        gg, uu = want[t] @ wg.T, want[t] @ wu.T
        hh = gg / (1 + np.exp(-gg)) * uu
        gate = f64(L.gates).reshape(N, K)[t, k][:, None]
        np.add.at(ref, t, gate * (hh @ wd.T))
        ag, au = np.abs(want[t]) @ np.abs(wg).T, np.abs(want[t]) @ np.abs(wu).T
        np.add.at(mag, t, gate * ((1.1 * ag * np.abs(uu) + np.abs(gg) * au + np.abs(hh)) @ np.abs(wd).T))
    # 2^-4 each from x and the weights, with the small codes' share and second order: 0.25 of the magnitudes
    assert (np.abs(f64(L.y) - ref) <= 0.25 * mag).all()
    rel = np.linalg.norm(f64(L.y) - ref) / np.linalg.norm(ref)
    # independent roundings, uniform within half a step of 2^-4 at most: rms 2^-4 / sqrt(3) = 0.036 a factor, and five
    # factors (x and weight twice, h once): 0.08 in quadrature if all were at the largest step
    print(f"[chain] relative distance from the layer in 64 bits: {rel:.4f}")
    assert rel < 0.081


def test_chain_captured_and_replayed():
    print("[case] graph of the 8-bit chain", flush=True)
    L = Layer(seed=1)
    want = {}
    for seed in (0, 1, 2):
        L.load(seed)
        L.forward()
        L.backward()
        torch.cuda.synchronize()
        want[seed] = L.snapshot()
    assert not np.array_equal(want[0]["slot_of"], want[1]["slot_of"])
    L.load(0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.forward()
        L.backward()
    for i in range(6):
        seed = i % 3
        L.load(seed)
        noise = torch.randn(512, 512, device="cuda") @ torch.randn(512, 512, device="cuda")
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k, v in L.snapshot().items():
            np.testing.assert_array_equal(v, want[seed][k], err_msg=f"replay {i}: {k}")
        del noise


def test_two_chains_at_once():
    """Two layers with buffers of their own on two streams, and one stream handed in for the calls of another."""
    print("[case] two streams", flush=True)
    layers = [Layer(seed=2), Layer(R=2, E=8, S=53, K=3, H=528, F=144, B=1, seed=3, score=mx.SCORE_SOFTMAX, groups=1)]
    want = []
    for L in layers:
        L.load(5)
        L.forward()
        L.backward()
        torch.cuda.synchronize()
        want.append(L.snapshot())
        L.load(5)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(3):
        for L, st in zip(layers, streams):
            with torch.cuda.stream(st):
                L.forward()
                L.backward()
    torch.cuda.synchronize()
    for L, w in zip(layers, want):
        for k, v in L.snapshot().items():
            np.testing.assert_array_equal(v, w[k], err_msg=k)
    # the stream argument: enqueued there, whatever stream is current
    L, s = layers[0], layers[0].s
    L.load(6)
    torch.cuda.synchronize()
    mx.moonep_rmsnorm_quant(s, L.x, L.res, L.norm_w, 1e-6, L.res_out, L.y16, L.y8, L.ys, stream=streams[1])
    streams[1].synchronize()
    got = L.y8.view(torch.uint8).cpu().numpy().copy()
    mx.moonep_rmsnorm_quant(s, L.x, L.res, L.norm_w, 1e-6, L.res_out, L.y16, L.y8, L.ys)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(L.y8.view(torch.uint8).cpu().numpy(), got)


def test_refuses_wrong_tensors():
    L = Layer(seed=4)
    L.load(0)
    call = lambda **k: mx.moonep_dispatch_quant(L.s, **{**dict(x8=L.y8, xs=L.ys, slot_of=L.b.slot_of, buf8=L.buf8,  # noqa: E731
                                                               bufs=L.bufs), **k})
    with pytest.raises(ValueError, match="GPU"):
        call(x8=L.y8.cpu())
    with pytest.raises(ValueError, match="dtype"):
        call(x8=L.y8.view(torch.int8))
    with pytest.raises(ValueError, match="elements"):
        call(bufs=L.bufs[:-1])
    with pytest.raises(ValueError, match="contiguous"):
        call(buf8=torch.empty((L.s.H, L.s.NK), dtype=torch.uint8, device="cuda").t())
    with pytest.raises(mx.MoonepError) as e:
        call(xs=None)
    assert e.value.code == -2
    with pytest.raises(mx.MoonepError) as e:
        mx.moonep_router(L.s, L.opts, L.logits, L.topk, L.gates, L.counts, L.prob, L.loss, L.ws[:64])
    assert e.value.code == -4
    with pytest.raises(mx.MoonepError):
        mx.moonep_router(L.s, L.opts, L.logits, L.topk, L.gates, counts=L.counts)
