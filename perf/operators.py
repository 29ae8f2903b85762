"""The router and the 8-bit expert path, as cases to be measured.

Each case is one pass through one operator on one GPU.  With `own` false, run()
computes the operator in its plain form, elementary torch operations in fp32
(fp64 for sums over all tokens); with `own` true it makes the calls of
load_balancing_amd that a user's program makes.  exact() computes the same
outputs in fp64 from the operator's definition.

Kinds of cases:
  router      ids, gates, counts and the balance loss from router logits
  router_bwd  their gradient with respect to the logits
  norm        residual addition, RMS norm and its 8-bit output with scales
  dispatch    8-bit rows and their scales into the expert-grouped buffer
  weights     bf16 expert matrices to 8 bits with a scale per 128 x 128 block
  glu, gemm   the experts' products over the grouped buffer: gate and up with
              the activation and an 8-bit output; one projection with bf16 output

8-bit values are OCP e4m3 codes with one E8M0 scale (a power of two) per block
of 128 along a row; rows of scales are padded to whole groups of four bytes
with ones.
"""
import math

import torch

own = False

SOFTMAX, SIGMOID = 0, 1
BLOCK = 128


def listed():
    return [
        # serving: eight tokens on each of 8 ranks take their experts, no loss
        dict(name="router_decode", kind="router", R=8, E=64, S=8, K=8, score=SOFTMAX, normalize=True, scale=1.0,
             groups=1, bf16=False, loss=False),
        # training: one microbatch of the DeepSeek-V3-like shape, loss per rank
        dict(name="router_train", kind="router", R=32, E=256, S=4096, K=8, score=SIGMOID, normalize=True, scale=2.5,
             groups=32, bf16=False, loss=True),
        # its backward on the 128-expert shape, bf16 logits, loss over all tokens
        dict(name="router_bwd", kind="router_bwd", R=16, E=128, S=8192, K=8, score=SOFTMAX, normalize=False, scale=1.0,
             groups=1, bf16=True, loss=True),
        # one decoding step's rows before a wide layer
        dict(name="norm_decode", kind="norm", N=8, H=7168, res=True, y=True),
        # prefill or a training microbatch, 4096 wide
        dict(name="norm_prefill", kind="norm", N=131072, H=4096, res=True, y=True),
        # a few tokens a rank into the grouped buffer
        dict(name="dispatch_decode", kind="dispatch", R=8, E=64, S=13, K=8, H=2048, skew=0.5),
        # the sweep shape
        dict(name="dispatch_sweep", kind="dispatch", R=8, E=64, S=4096, K=8, H=2048, skew=0.5),
        # a small model's experts, ragged against the blocks
        dict(name="weights_small", kind="weights", E=16, out=208, inp=336),
        # one projection of the sweep shape's 64 experts
        dict(name="weights_sweep", kind="weights", E=64, out=1408, inp=2048),
        # gate and up for 32 decoding tokens: about four rows an expert
        dict(name="glu_decode", kind="glu", R=8, E=64, S=4, K=8, inp=2048, out=1408, B=3, skew=0.5),
        # gate and up on the sweep shape, its replicas in the training slots
        dict(name="glu_sweep", kind="glu", R=8, E=64, S=4096, K=8, inp=2048, out=1408, B=8, skew=0.5),
        # down for a chunk of a prompt: ragged segments of a few hundred rows
        dict(name="down_chunk", kind="gemm", R=8, E=64, S=509, K=8, inp=1408, out=2048, B=3, skew=0.5),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["router", "router_bwd", "norm", "dispatch", "weights", "glu", "gemm"])
    R = rng.choice([1, 2, 4, 8, 16, 32])
    E = min(R * rng.randint(2, 16), 384)
    E -= E % R
    K = rng.randint(1, min(8, E))
    if kind in ("router", "router_bwd"):
        S = _log_int(rng, 1, min(8192, 131072 * 128 // (R * E)))
        return dict(kind=kind, R=R, E=E, S=S, K=K, score=rng.choice([SOFTMAX, SIGMOID]), normalize=rng.random() < 0.5,
                    scale=rng.choice([1.0, 2.5]), groups=rng.choice([1, R]), bf16=rng.random() < 0.5,
                    loss=kind == "router_bwd" or rng.random() < 0.7)
    if kind == "norm":
        H = 16 * _log_int(rng, 4, 512)
        return dict(kind=kind, N=_log_int(rng, 1, 131072 * 4096 // max(H, 4096)), H=H, res=rng.random() < 0.8,
                    y=rng.random() < 0.7)
    if kind == "dispatch":
        H = 16 * _log_int(rng, 4, 448)
        S = _log_int(rng, 1, max(1, min(8192, 32768 * 8 * 2048 // (R * K * max(H, 1024)))))
        return dict(kind=kind, R=R, E=E, S=S, K=K, H=H, skew=rng.choice([0.0, 0.5, 1.5]))
    if kind == "weights":
        out, inp = 16 * _log_int(rng, 4, 256), 16 * _log_int(rng, 4, 256)
        return dict(kind=kind, E=_log_int(rng, 1, max(1, min(128, 64 * 1408 * 2048 // (out * inp)))), out=out, inp=inp)
    out, inp = 16 * _log_int(rng, 8, 192), 16 * _log_int(rng, 8, 192)
    most = 262144 * 2 * 1408 * 2048 // (2 * (2 if kind == "glu" else 1) * out * inp * R * K)
    S = _log_int(rng, 1, max(1, min(2048, most)))
    return dict(kind=kind, R=R, E=E, S=S, K=K, inp=inp, out=out, B=rng.randint(0, 4),
                skew=rng.choice([0.0, 0.5, 1.5]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def scale_bytes(cols):
    return 4 * (-(-cols // (4 * BLOCK)))


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(shape, g, std=1.0):
    return torch.randn(shape, generator=g, device="cuda") * std


def _logits(R, E, S, skew, g):
    """Router logits: a preference of the layer for some experts, and each token's own."""
    return _normal((R * S, E), g) + skew * _normal((E,), g)


def _plan(R, E, S, K, counts):
    """The plan table of moonep_plan for these expert counts (greedy, lowest id
    first), as int32 words, and the number of its replicas."""
    C, L = S * K, E // R
    load = [sum(counts[r * L:(r + 1) * L]) for r in range(R)]
    spill = [0] * E
    for r in range(R):
        over = max(0, load[r] - C)
        for e in range(r * L, (r + 1) * L):
            spill[e] = min(counts[e], over)
            over -= spill[e]
    room = [max(0, C - x) for x in load]
    reps, d = [], 0
    for e in range(E):
        left = spill[e]
        while left:
            while not room[d]:
                d += 1
            n = min(left, room[d])
            reps.append((e, d, n, spill[e] - left))
            room[d] -= n
            left -= n
    keep = [counts[e] - spill[e] for e in range(E)]
    home_off, at = [0] * E, [0] * R
    for e in range(E):
        home_off[e] = at[e // L]
        at[e // L] += keep[e]
    row_off = []
    for _, d, n, _ in reps:
        row_off.append(at[d])
        at[d] += n
    cap = E + R
    pad = lambda v, n: list(v) + [0] * (n - len(v))  # noqa: E731
    first, cnt = [0] * E, [0] * E
    for j, (e, _, _, _) in enumerate(reps):
        first[e] = first[e] if cnt[e] else j
        cnt[e] += 1
    rfirst, rcnt = [0] * R, [0] * R
    for j, (_, d, _, _) in enumerate(reps):
        rfirst[d] = rfirst[d] if rcnt[d] else j
        rcnt[d] += 1
    spilling = [e for e in range(E) if cnt[e]]
    header = [len(reps), len(spilling), sum(x < C for x in load), max(rcnt), max(counts), C, L, cap] + [0] * 8
    words = header
    for i in (0, 1, 2, 3):
        words = words + pad([r[i] for r in reps], cap)
    words = words + pad(row_off, cap) + spill + keep + home_off + first + cnt + pad(spilling, E) + load + rfirst + rcnt
    return words, reps, row_off, keep, home_off


def _routing(case, g):
    """ids, and the plan, replica weight slots and slot map they lead to."""
    R, E, S, K = case["R"], case["E"], case["S"], case["K"]
    ids = torch.topk(_logits(R, E, S, case["skew"], g), K, dim=1).indices.reshape(-1)
    counts = torch.bincount(ids, minlength=E)
    words, reps, row_off, keep, home_off = _plan(R, E, S, K, counts.tolist())
    C, L, B = S * K, E // R, case.get("B", 0)
    hosted, wslot = [0] * R, [-1] * (E + R)
    for j, (_, d, _, _) in enumerate(reps):
        wslot[j] = d * B + hosted[d] if hosted[d] < B else -1
        hosted[d] += 1
    # entry i of expert e (in token order) sits in the home rows or in the replica that covers i
    order = torch.sort(ids, stable=True).indices
    pieces = [(e, 0, keep[e], (e // L) * C + home_off[e]) for e in range(E)]
    pieces += [(e, keep[e] + so, n, d * C + ro) for (e, d, n, so), ro in zip(reps, row_off)]
    pieces = sorted(p for p in pieces if p[2])
    n = torch.tensor([p[2] for p in pieces], device="cuda")
    row0 = torch.tensor([p[3] for p in pieces], device="cuda")
    rows = torch.repeat_interleave(row0 - (torch.cumsum(n, 0) - n), n) + torch.arange(ids.numel(), device="cuda")
    slot_of = torch.empty_like(ids)
    slot_of[order] = rows  # pieces ascend by expert and place, as `order` does
    return dict(ids=ids.int(), plan=torch.tensor(words, dtype=torch.int32, device="cuda"), n_rep=len(reps),
                wslot=torch.tensor(wslot, dtype=torch.int32, device="cuda"), slot_of=slot_of.int(),
                longest=max(p[2] for p in pieces), reps=reps)


def _random_codes(rows, cols, g):
    """Rows of a normed activation in 8 bits with their scales, as the layer before leaves them."""
    x = _normal((rows, cols), g)
    return _plain_quant_rows(x)


def _weight_rows(E, mats, g):
    """[E, stride] bytes: each expert's matrices in 8 bits, codes then scales, and the offsets of both."""
    at, offs = 0, []
    for out, inp in mats:
        code, at = at, at + out * inp
        at += -at % 4
        scale, at = at, at + -(-out // BLOCK) * scale_bytes(inp)
        at += -at % 16
        offs.append((code, scale))
    rows = torch.zeros((E, at), dtype=torch.uint8, device="cuda")
    for e in range(E):
        for (out, inp), (code, scale) in zip(mats, offs):
            c, s = _plain_quant_blocks((_normal((1, out, inp), g) * inp ** -0.5).bfloat16().float())
            rows[e, code:code + out * inp] = c.view(torch.uint8).reshape(-1)
            rows[e, scale:scale + s.numel()] = s.reshape(-1)
    return rows, offs


def prepare(case, seed):
    g = _gen(seed)
    kind = case["kind"]
    st = dict(case)
    dev = "cuda"
    if kind in ("router", "router_bwd"):
        R, E, S, K, G = case["R"], case["E"], case["S"], case["K"], case["groups"]
        t = torch.bfloat16 if case["bf16"] else torch.float32
        st["logits"] = _logits(R, E, S, 0.5, g).to(t)
        st["topk_idx"] = torch.empty(R * S * K, dtype=torch.int32, device=dev)
        st["gates"] = torch.empty(R * S * K, dtype=torch.float32, device=dev)
        st["counts"] = torch.empty((G, E), dtype=torch.int32, device=dev)
        st["prob_sum"] = torch.empty((G, E), dtype=torch.float32, device=dev)
        st["loss_out"] = torch.empty(1, dtype=torch.float32, device=dev)
        st["workspace"] = torch.empty(8 * (E + 64) * (4096 + 2 * G), dtype=torch.uint8, device=dev)
        if kind == "router_bwd":
            st["topk_idx"] = torch.sort(st["logits"], dim=1, descending=True, stable=True).indices[:, :K].int().reshape(-1)
            one = torch.ones(R * S * K, dtype=torch.int64, device=dev)
            grp = torch.arange(R * S * K, device=dev) // (R * S * K // G)
            st["counts"] = torch.zeros(G * E, dtype=torch.int64, device=dev).index_add_(
                0, grp * E + st["topk_idx"], one).int().view(G, E)
            st["d_gates"] = _normal((R * S * K,), g, 0.1)
            st["d_loss"] = torch.full((1,), 0.01, device=dev) * (1 + 0.1 * _normal((1,), g).abs())
            st["d_logits"] = torch.empty_like(st["logits"])
    elif kind == "norm":
        N, H = case["N"], case["H"]
        st["x"] = _normal((N, H), g).bfloat16()
        st["resid"] = (_normal((N, H), g, 3.0)).bfloat16() if case["res"] else None
        st["weight"] = (1 + _normal((H,), g, 0.2)).bfloat16()
        st["eps"] = 1e-6
        st["res_out"] = torch.empty_like(st["x"]) if case["res"] else None
        st["y_out"] = torch.empty_like(st["x"]) if case["y"] else None
        st["y8"] = torch.empty((N, H), dtype=torch.float8_e4m3fn, device=dev)
        st["ys"] = torch.empty((N, scale_bytes(H)), dtype=torch.uint8, device=dev)
    elif kind == "dispatch":
        N, H, K = case["R"] * case["S"], case["H"], case["K"]
        st.update(_routing(case, g))
        st["x8"], st["xs"] = _random_codes(N, H, g)
        st["buf8"] = torch.empty((N * K, H), dtype=torch.float8_e4m3fn, device=dev)
        st["bufs"] = torch.empty((N * K, scale_bytes(H)), dtype=torch.uint8, device=dev)
    elif kind == "weights":
        E, out, inp = case["E"], case["out"], case["inp"]
        st["w"] = torch.randn((E, out * inp), generator=g, device=dev, dtype=torch.bfloat16) * inp ** -0.5
        code = out * inp
        stride = code + -(-out // BLOCK) * scale_bytes(inp)
        stride += -stride % 16
        st["stride"] = stride
        st["w8"] = torch.zeros((E, stride), dtype=torch.uint8, device=dev)
    else:
        NK = case["R"] * case["S"] * case["K"]
        E, R, B, inp, out = case["E"], case["R"], case["B"], case["inp"], case["out"]
        st.update(_routing(case, g))
        st["x8"], st["xs"] = _random_codes(NK, inp, g)
        st["w_home"], st["offs"] = _weight_rows(E, [(out, inp)] * (2 if kind == "glu" else 1), g)
        st["pool"] = torch.zeros((R * B, st["w_home"].shape[1]), dtype=torch.uint8, device=dev)
        for j, w in enumerate(st["wslot"].tolist()):
            if w >= 0:
                st["pool"][w] = st["w_home"][st["reps"][j][0]]
        if kind == "glu":
            st["h8"] = torch.empty((NK, out), dtype=torch.float8_e4m3fn, device=dev)
            st["hs"] = torch.empty((NK, scale_bytes(out)), dtype=torch.uint8, device=dev)
        else:
            st["y_out"] = torch.empty((NK, out), dtype=torch.bfloat16, device=dev)
    return st


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _scale_byte(amax):
    """Least power of two that brings amax to at most 448, as its E8M0 byte; 127 for an empty block."""
    b = ((amax.view(torch.int32) + 0x1FFFFF) >> 23) - 8
    b = torch.where(amax == 0, 127, b.clamp(min=1))
    return torch.where(torch.isfinite(amax), b, 255)


def _inverse(byte):
    """1 / 2^(byte - 127): a product with it is exact, where a division need not be."""
    return (254 - byte).to(torch.uint8).view(torch.float8_e8m0fnu).float()


def _plain_quant_rows(y):
    """[rows, cols] fp32 -> e4m3 codes and [rows, scale_bytes(cols)] E8M0 bytes, one for each 128 columns."""
    rows, cols = y.shape
    nb = -(-cols // BLOCK)
    p = torch.nn.functional.pad(y, (0, nb * BLOCK - cols)).view(rows, nb, BLOCK)
    byte = _scale_byte(p.abs().amax(2))
    codes = (p * _inverse(byte)[:, :, None]).view(rows, -1)[:, :cols].to(torch.float8_e4m3fn)
    scales = torch.full((rows, scale_bytes(cols)), 127, dtype=torch.uint8, device=y.device)
    scales[:, :nb] = byte.to(torch.uint8)
    return codes.contiguous(), scales


def _plain_quant_blocks(w):
    """[n, out, in] fp32 -> e4m3 codes and [n, ceil(out / 128), scale_bytes(in)] E8M0 bytes of 128 x 128 blocks."""
    n, out, inp = w.shape
    ob, ib = -(-out // BLOCK), -(-inp // BLOCK)
    p = torch.nn.functional.pad(w, (0, ib * BLOCK - inp, 0, ob * BLOCK - out)).view(n, ob, BLOCK, ib, BLOCK)
    byte = _scale_byte(p.abs().amax((2, 4)))
    codes = (p * _inverse(byte)[:, :, None, :, None]).view(n, ob * BLOCK, ib * BLOCK)[:, :out, :inp]
    scales = torch.full((n, ob, scale_bytes(inp)), 127, dtype=torch.uint8, device=w.device)
    scales[:, :, :ib] = byte.to(torch.uint8)
    return codes.to(torch.float8_e4m3fn).contiguous(), scales


def _e8m0(s):
    return s.view(torch.float8_e8m0fnu)


def _plain_scores(st):
    l = st["logits"].float()
    if st["score"] == SOFTMAX:
        s = torch.exp(l - l.amax(1, keepdim=True))
        return s, s.sum(1, keepdim=True)
    s = 1 / (1 + torch.exp(-l))
    return s, s.sum(1, keepdim=True) + 1e-20


def _plain_router(st):
    E, K, G = st["E"], st["K"], st["groups"]
    N = st["logits"].shape[0]
    s, Z = _plain_scores(st)
    idx = torch.sort(st["logits"], dim=1, descending=True, stable=True).indices[:, :K]
    top = torch.gather(s, 1, idx)
    if st["normalize"]:
        top = top / (top.sum(1, keepdim=True) + (1e-20 if st["score"] == SIGMOID else 0.0))
    elif st["score"] == SOFTMAX:
        top = top / Z
    ids, gates = idx.int().reshape(-1), (top * st["scale"]).reshape(-1)
    if not st["loss"]:
        return dict(ids=ids, gates=gates)
    P = (s / Z).double().view(G, N // G, E).sum(1)
    T = torch.zeros((G, E), dtype=torch.int64, device=s.device).scatter_add_(
        1, idx.reshape(G, -1), torch.ones_like(idx).reshape(G, -1))
    loss = (T * P).sum(1).mean() * E / (K * (N // G) ** 2)
    return dict(ids=ids, gates=gates, counts=T.int(), prob_sum=P.float(), loss=loss.float().view(1))


def _plain_router_bwd(st):
    E, K, G, c = st["E"], st["K"], st["groups"], st["scale"]
    N = st["logits"].shape[0]
    n = N // G
    s, Z = _plain_scores(st)
    idx, dg = st["topk_idx"].long().view(N, K), st["d_gates"].view(N, K)
    a = (st["d_loss"] * E / (K * float(n) * n * G) * st["counts"].float()).repeat_interleave(n, 0)
    ds = (a - (a * s / Z).sum(1, keepdim=True)) / Z
    top = torch.gather(s, 1, idx)
    if st["normalize"]:
        W = top.sum(1, keepdim=True) + (1e-20 if st["score"] == SIGMOID else 0.0)
        part = c * (dg - (dg * top / W).sum(1, keepdim=True)) / W
    elif st["score"] == SOFTMAX:
        part = c * dg / Z
        ds = ds - c * (dg * top / Z).sum(1, keepdim=True) / Z
    else:
        part = c * dg
    ds = ds.scatter_add(1, idx, part)
    dl = ds * s if st["score"] == SOFTMAX else ds * s * (1 - s)
    return dl.to(st["logits"].dtype)


def _plain_norm(st):
    r = st["x"] if st["resid"] is None else (st["x"].float() + st["resid"].float()).bfloat16()
    v = r.float()
    y = v * torch.rsqrt((v * v).mean(1, keepdim=True) + st["eps"]) * st["weight"].float()
    y8, ys = _plain_quant_rows(y)
    out = dict(y8=y8, ys=_e8m0(ys))
    if st["resid"] is not None:
        out["res"] = r
    if st["y"]:
        out["y"] = y.bfloat16()
    return out


def _plain_dispatch(st):
    slot = st["slot_of"].long()
    x8, xs = st["x8"].view(torch.uint8), st["xs"]
    buf8, bufs = torch.empty_like(st["buf8"]).view(torch.uint8), torch.empty_like(st["bufs"])
    buf8[slot] = x8.repeat_interleave(st["K"], 0)
    bufs[slot] = xs.repeat_interleave(st["K"], 0)
    return dict(rows=buf8.view(torch.float8_e4m3fn), scales=_e8m0(bufs))


def _plain_weights(st):
    E, out, inp = st["E"], st["out"], st["inp"]
    codes, scales = _plain_quant_blocks(st["w"].view(E, out, inp).float())
    return dict(codes=codes, scales=_e8m0(scales))


def _expand(s, cols):
    return s.view(torch.float8_e8m0fnu).float().repeat_interleave(BLOCK, -1)[..., :cols]


def _plain_products(st):
    """The grouped products in fp32, every segment of the plan padded to the longest: one product per matrix of the expert."""
    R, E, S, K, inp, out = (st[k] for k in ("R", "E", "S", "K", "inp", "out"))
    C, cap, nr, p = S * K, E + R, st["n_rep"], st["plan"].long()
    rep = [p[16 + i * cap:16 + i * cap + nr] for i in range(5)]  # expert, host, count, offset among the spilled, first row
    keep, home_off = p[16 + 5 * cap + E:16 + 5 * cap + 2 * E], p[16 + 5 * cap + 2 * E:16 + 5 * cap + 3 * E]
    e = torch.arange(E, device=p.device)
    row0 = torch.cat([e // (E // R) * C + home_off, rep[1] * C + rep[4]])
    n = torch.cat([keep, rep[2]])
    ws = st["wslot"].long()[:nr]
    source = torch.cat([e, torch.where(ws >= 0, E + ws, rep[0])])
    seg = torch.repeat_interleave(torch.arange(E + nr, device=p.device), n)
    pos = torch.arange(R * C, device=p.device) - (torch.cumsum(n, 0) - n)[seg]
    row = row0[seg] + pos
    x = st["x8"].float() * _expand(st["xs"], inp)
    xp = torch.zeros((E + nr, st["longest"], inp), device=p.device)
    xp[seg, pos] = x[row]
    weights = torch.cat([st["w_home"], st["pool"]])[source]

    def product(code, scale):
        w = weights[:, code:code + out * inp].view(torch.float8_e4m3fn).reshape(-1, out, inp).float()
        sc = weights[:, scale:scale + -(-out // BLOCK) * scale_bytes(inp)].reshape(E + nr, -1, scale_bytes(inp))
        w = w * _expand(sc, inp).repeat_interleave(BLOCK, 1)[:, :out]
        y = torch.empty((R * C, out), device=p.device)
        y[row] = torch.bmm(xp, w.transpose(1, 2).contiguous())[seg, pos]
        return y

    if st["kind"] == "gemm":
        return dict(y=product(*st["offs"][0]).bfloat16())
    gate, up = product(*st["offs"][0]), product(*st["offs"][1])
    h8, hs = _plain_quant_rows(gate / (1 + torch.exp(-gate)) * up)
    return dict(h8=h8, hs=_e8m0(hs))


_PLAIN = dict(router=_plain_router, router_bwd=_plain_router_bwd, norm=_plain_norm, dispatch=_plain_dispatch,
              weights=_plain_weights, glu=_plain_products, gemm=_plain_products)


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------

def _own(st):
    import load_balancing_amd as mx

    kind = st["kind"]
    if kind == "norm":
        s = mx.Shape(1, 1, st["N"], 1, st["H"])
        mx.moonep_rmsnorm_quant(s, st["x"], st["resid"], st["weight"], st["eps"], st["res_out"], st["y_out"], st["y8"],
                                st["ys"])
        out = dict(y8=st["y8"], ys=_e8m0(st["ys"]))
        if st["resid"] is not None:
            out["res"] = st["res_out"]
        if st["y"]:
            out["y"] = st["y_out"]
        return out
    if kind == "weights":
        E, out, inp, stride = st["E"], st["out"], st["inp"], st["stride"]
        s = mx.Shape(1, E, 0, 1, 16)
        mx.moonep_quant_weights(s, inp, out, st["w"], out * inp, 0, st["w8"], stride, 0, out * inp)
        n = -(-out // BLOCK) * scale_bytes(inp)
        return dict(codes=st["w8"][:, :out * inp].view(torch.float8_e4m3fn).view(E, out, inp),
                    scales=_e8m0(st["w8"][:, out * inp:out * inp + n]).unflatten(1, (-1, scale_bytes(inp))))
    s = mx.Shape(st["R"], st["E"], st["S"], st["K"], st.get("H", 16))
    if kind in ("router", "router_bwd"):
        opts = mx.RouterOpts(st["score"], st["normalize"], st["groups"], st["bf16"], st["scale"])
        if kind == "router_bwd":
            mx.moonep_router_bwd(s, opts, st["logits"], st["topk_idx"], st["counts"], st["d_gates"], st["d_loss"],
                                 st["d_logits"])
            return st["d_logits"]
        if not st["loss"]:
            mx.moonep_router(s, opts, st["logits"], st["topk_idx"], st["gates"])
            return dict(ids=st["topk_idx"], gates=st["gates"])
        mx.moonep_router(s, opts, st["logits"], st["topk_idx"], st["gates"], st["counts"], st["prob_sum"],
                         st["loss_out"], st["workspace"])
        return dict(ids=st["topk_idx"], gates=st["gates"], counts=st["counts"], prob_sum=st["prob_sum"],
                    loss=st["loss_out"])
    if kind == "dispatch":
        mx.moonep_dispatch_quant(s, st["x8"], st["xs"], st["slot_of"], st["buf8"], st["bufs"])
        return dict(rows=st["buf8"], scales=_e8m0(st["bufs"]))
    stride = st["w_home"].shape[1]
    if kind == "glu":
        (gc, gs), (uc, us) = st["offs"]
        mx.moonep_expert_glu_quant(s, st["plan"], st["wslot"], st["B"], st["inp"], st["out"], st["x8"], st["xs"],
                                   st["w_home"], st["pool"], stride, gc, gs, uc, us, st["h8"], st["hs"])
        return dict(h8=st["h8"], hs=_e8m0(st["hs"]))
    code, scale = st["offs"][0]
    mx.moonep_expert_gemm_quant(s, st["plan"], st["wslot"], st["B"], st["inp"], st["out"], st["x8"], st["xs"],
                                st["w_home"], st["pool"], stride, code, scale, st["y_out"])
    return dict(y=st["y_out"])


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["kind"]](state)


def work(case):
    kind = case["kind"]
    if kind in ("router", "router_bwd"):
        N, E, K = case["R"] * case["S"], case["E"], case["K"]
        size = 2 if case["bf16"] else 4
        table = case["groups"] * E
        if kind == "router":
            return dict(bytes=N * E * size + N * K * 8 + (8 * table + 4 if case["loss"] else 0), flops=6 * N * E)
        return dict(bytes=2 * N * E * size + N * K * 8 + 4 * table + 4, flops=12 * N * E)
    if kind == "norm":
        N, H = case["N"], case["H"]
        return dict(bytes=N * (H * (2 + (4 if case["res"] else 0) + (2 if case["y"] else 0) + 1) + scale_bytes(H)) + 2 * H,
                    flops=8 * N * H)
    if kind == "dispatch":
        N, K, row = case["R"] * case["S"], case["K"], case["H"] + scale_bytes(case["H"])
        return dict(bytes=N * row + N * K * (row + 4), flops=0)
    if kind == "weights":
        n = case["E"] * case["out"] * case["inp"]
        return dict(bytes=3 * n + case["E"] * -(-case["out"] // BLOCK) * scale_bytes(case["inp"]), flops=2 * n)
    NK, inp, out = case["R"] * case["S"] * case["K"], case["inp"], case["out"]
    mats = 2 if kind == "glu" else 1
    weights = min(case["E"], NK) * mats * out * inp  # each chosen expert's once; fewer where rows share experts
    written = out + scale_bytes(out) if kind == "glu" else 2 * out
    return dict(bytes=weights + NK * (inp + scale_bytes(inp) + written), flops=2 * mats * NK * inp * out)


# ---------------------------------------------------------------------------
# the definitions in fp64
# ---------------------------------------------------------------------------

def _two(k):
    """2^k in fp64 for whole k, exactly."""
    return ((k.long() + 1023) << 52).view(torch.float64)


def _code64(v):
    """fp64 -> the nearest e4m3 value (ties to even), |v| <= 448."""
    ex = torch.frexp(v)[1].clamp(min=-5) - 4  # quantum 2^ex: 3 bits after the leading one, 2^-9 at least
    return torch.round(v * _two(-ex)) * _two(ex)


def _quant64(y, tile):
    """Codes and scales of [n, out, in] in fp64, one scale for each tile[0] x tile[1] block."""
    n, out, inp = y.shape
    ob, ib = -(-out // tile[0]), -(-inp // tile[1])
    p = y.new_zeros((n, ob * tile[0], ib * tile[1]))
    p[:, :out, :inp] = y
    amax = p.view(n, ob, tile[0], ib, tile[1]).abs().amax((2, 4))
    ex = torch.frexp(amax / 448)[1].clamp(min=-126)  # amax / 448 is in [2^(ex - 1), 2^ex)
    ex = torch.where(amax <= 448 * _two(ex - 1), ex - 1, ex).clamp(min=-126)
    scale = torch.where(amax == 0, torch.ones_like(amax), _two(ex))
    per = scale.repeat_interleave(tile[0], 1).repeat_interleave(tile[1], 2)[:, :out, :inp]
    padded = y.new_ones((n, ob, scale_bytes(inp)))
    padded[:, :, :ib] = scale
    return _code64(y / per), padded


def _value64(codes, scales):
    s = _two(scales.long() - 127)
    return codes.double() * s.repeat_interleave(BLOCK, 1)[:, :codes.shape[1]]


def _exact_products(st):
    R, E, K, inp, out = st["R"], st["E"], st["K"], st["inp"], st["out"]
    C, L = st["S"] * K, E // R
    words = st["plan"].tolist()
    cap = E + R
    part = lambda i, n, at=16 + 5 * cap: words[at + i * E:at + i * E + n]  # noqa: E731
    segs = [((e // L) * C + o, n, e, False) for e, (n, o) in enumerate(zip(part(1, E), part(2, E)))]
    for j, (e, d, n, _) in enumerate(st["reps"]):
        w = int(st["wslot"][j])
        segs.append((d * C + words[16 + 4 * cap + j], n, e if w < 0 else w, w >= 0))
    got = [torch.zeros((R * C, out), dtype=torch.float64, device="cuda") for _ in st["offs"]]
    for row0, n, at, pooled in segs:
        if not n:
            continue
        x = _value64(st["x8"][row0:row0 + n], st["xs"][row0:row0 + n])
        wrow = (st["pool"] if pooled else st["w_home"])[at]
        for y, (code, scale) in zip(got, st["offs"]):
            sc = wrow[scale:scale + -(-out // BLOCK) * scale_bytes(inp)].view(-1, scale_bytes(inp))
            w = _value64(wrow[code:code + out * inp].view(torch.float8_e4m3fn).view(out, inp),
                         sc.repeat_interleave(BLOCK, 0)[:out])
            y[row0:row0 + n] = x @ w.T
    if st["kind"] == "gemm":
        return dict(y=got[0])
    h, hs = _quant64((got[0] * torch.sigmoid(got[0]) * got[1])[None], (1, BLOCK))
    return dict(h8=h[0], hs=hs[0])


def _exact_router(st):
    """Both directions by autograd over the fp64 definition."""
    N, E, K, G, c = st["logits"].shape[0], st["E"], st["K"], st["groups"], st["scale"]
    n = N // G
    l = st["logits"].double().requires_grad_(st["kind"] == "router_bwd")
    tiny = 1e-20 if st["score"] == SIGMOID else 0.0
    s = torch.softmax(l, 1) if st["score"] == SOFTMAX else torch.sigmoid(l)
    p = s / (s.sum(1, keepdim=True) + tiny)
    # ids: order by value, then by id, through exact integer ranks of the logits
    rank = torch.unique(st["logits"].float(), return_inverse=True)[1]
    idx = torch.topk(rank * E + (E - 1 - torch.arange(E, device=l.device)), K, dim=1).indices
    top = s.gather(1, idx)
    gates = c * (top / (top.sum(1, keepdim=True) + tiny) if st["normalize"] else top)
    T = torch.nn.functional.one_hot(idx, E).view(G, n * K, E).sum(1)
    P = p.view(G, n, E).sum(1)
    loss = (T * P).sum() * E / (K * n * n * G)
    if st["kind"] == "router_bwd":
        total = (gates.reshape(-1) * st["d_gates"].double()).sum() + loss * st["d_loss"].double()[0]
        return torch.autograd.grad(total, l)[0]
    out = dict(ids=None, gates=gates.reshape(-1))
    if st["loss"]:
        out.update(counts=None, prob_sum=P, loss=loss.view(1))
    return out


def exact(case, seed):
    st = prepare(case, seed)
    kind = case["kind"]
    if kind in ("router", "router_bwd"):
        return _exact_router(st)
    if kind == "norm":
        r = st["x"].double()
        if st["resid"] is not None:
            r = (r + st["resid"].double()).float().bfloat16().double()
        y = r / torch.sqrt((r * r).mean(1, keepdim=True) + st["eps"]) * st["weight"].double()
        y8, ys = _quant64(y[:, None], (1, BLOCK))
        out = dict(y8=y8[:, 0], ys=ys[:, 0])
        if st["resid"] is not None:
            out["res"] = r
        if case["y"]:
            out["y"] = y
        return out
    if kind == "dispatch":
        src = torch.empty_like(st["slot_of"], dtype=torch.int64)
        src[st["slot_of"].long()] = torch.arange(src.numel(), device=src.device)
        src = src // case["K"]
        return dict(rows=st["x8"].float()[src], scales=_two(st["xs"].long() - 127)[src])
    if kind == "weights":
        codes, scales = _quant64(st["w"].double().view(case["E"], case["out"], case["inp"]), (BLOCK, BLOCK))
        return dict(codes=codes, scales=scales)
    return _exact_products(st)
