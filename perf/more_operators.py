"""The experts' gradients, low-rank adapters and gradient clipping, as cases to be measured.

Each case is one pass through one operator on one GPU.  With `own` false, run()
computes the operator in its plain form, elementary torch operations in fp32
(fp64 for the sum of squares over all gradients); with `own` true it makes the
calls of load_balancing_amd that a user's program makes.  exact() computes the
same outputs in fp64 from the operator's definition.

Kinds of cases:
  dx           gradient of an expert projection's input rows, grouped by expert
  dw           gradient of its weights, per home expert and per replica, in fp32
  adapter      y = base + s (x A^T) B^T with each row's own low-rank adapter
  adapter_bwd  the gradients of its input and of every adapter
  clip         the norm over many gradient tensors, and their clipped values

An adapter's matrices A [rank, in] and B [out, rank] are one row of a bf16 bank.
"""
import math

import torch

own = False

GRAD_RUN = 16384  # elements of one entry of the gradient table, at most


def listed():
    return [
        # a short training microbatch: ragged segments of about 60 rows, down projection
        dict(name="dx_chunk", kind="dx", R=8, E=64, S=61, K=8, inp=1408, out=2048, B=8, skew=0.5),
        # the sweep shape, gate projection, its replicas in the training slots
        dict(name="dx_sweep", kind="dx", R=8, E=64, S=4096, K=8, inp=2048, out=1408, B=8, skew=0.5),
        # weight gradients of a short microbatch: writing them is most of the work
        dict(name="dw_chunk", kind="dw", R=8, E=64, S=61, K=8, inp=1408, out=2048, skew=0.5),
        # weight gradients on the sweep shape, one projection
        dict(name="dw_sweep", kind="dw", R=8, E=64, S=4096, K=8, inp=2048, out=1408, skew=0.5),
        # serving: one token of each of 16 requests, each with an adapter of its own
        dict(name="adapter_decode", kind="adapter", N=16, M=64, rank=16, inp=2048, out=2048, seqs=16, none=0.0,
             sorted=False),
        # serving: a ragged mix of prompts and single tokens, a part of them without an adapter
        dict(name="adapter_mixed", kind="adapter", N=1531, M=24, rank=32, inp=2048, out=1408, seqs=97, none=0.2,
             sorted=True),
        # prefill or a training microbatch, 4096 wide
        dict(name="adapter_prefill", kind="adapter", N=32768, M=8, rank=64, inp=4096, out=4096, seqs=40, none=0.1,
             sorted=False),
        # training on the same widths
        dict(name="adapter_bwd_train", kind="adapter_bwd", N=32768, M=4, rank=16, inp=4096, out=4096, seqs=40, none=0.0),
        # training many small tenants at once
        dict(name="adapter_bwd_tenants", kind="adapter_bwd", N=4099, M=32, rank=32, inp=2048, out=1408, seqs=151,
             none=0.1),
        # gradients of adapters: many small fp32 tensors
        dict(name="clip_adapters", kind="clip", tensors=448, least=32768, most=65536, bf16=False, odd=False, ratio=4.0),
        # bf16 gradients of a small model, biases and norms among them, odd sizes
        dict(name="clip_ragged", kind="clip", tensors=291, least=63, most=2097152, bf16=True, odd=True, ratio=3.0),
        # the sweep shape's experts, three matrices each
        dict(name="clip_experts", kind="clip", tensors=192, least=2883584, most=2883584, bf16=False, odd=False,
             ratio=8.0),
    ]


def _log_int(rng, lo, hi):
    hi = max(lo, hi)
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["dx", "dw", "adapter", "adapter_bwd", "clip"])
    if kind in ("dx", "dw"):
        R = rng.choice([1, 2, 4, 8, 16, 32])
        E = min(R * rng.randint(2, 16), 256)
        E -= E % R
        K = rng.randint(1, min(8, E))
        out, inp = 128 * _log_int(rng, 1, 22), 64 * _log_int(rng, 2, 44)
        while 4 * E * out * inp > 64 * 3 * 1408 * 2048 * 4:
            E -= R
        S = _log_int(rng, 1, min(4096, 262144 * 1408 * 2048 // (2 * out * inp * R * K)))
        case = dict(kind=kind, R=R, E=E, S=S, K=min(K, E), inp=inp, out=out, skew=rng.choice([0.0, 0.5, 1.5]))
        if kind == "dx":
            case["B"] = rng.randint(0, 4)
        return case
    if kind in ("adapter", "adapter_bwd"):
        rank = 8 * rng.choice([1, 1, 2, 2, 3, 4, 4, 5, 8, 8, 12, 16])
        out, inp = 8 * _log_int(rng, 8, 1024), 8 * _log_int(rng, 8, 1024)
        M = _log_int(rng, 1, min(256, 2 ** 26 // (rank * (out + inp))))
        N = _log_int(rng, 1, min(32768, 32768 * 8192 * 64 // ((out + inp) * max(rank, 64)), 2 ** 33 // (M * (out + inp))))
        case = dict(kind=kind, N=N, M=M, rank=rank, inp=inp, out=out, seqs=_log_int(rng, 1, N),
                    none=rng.choice([0.0, 0.1, 0.5]))
        if kind == "adapter":
            case["sorted"] = rng.random() < 0.5
        return case
    least = _log_int(rng, 1, 100000)
    most = _log_int(rng, least, 4000000)
    return dict(kind=kind, tensors=_log_int(rng, 1, min(1024, max(1, 2 ** 28 // most))), least=least, most=most,
                bf16=rng.random() < 0.5, odd=rng.random() < 0.5, ratio=rng.choice([0.5, 4.0]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(shape, g, std=1.0):
    return torch.randn(shape, generator=g, device="cuda") * std


def _bf16(shape, g, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16) * std


def _plan(R, E, C, counts):
    """The plan table of moonep_plan for these expert counts (greedy, lowest id
    first), as int32 words, and its segments: (expert, rank, rows, first row)
    of every home expert, then of every replica."""
    L = E // R
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
    words = [len(reps), len(spilling), sum(x < C for x in load), max(rcnt), max(counts), C, L, cap] + [0] * 8
    for i in (0, 1, 2, 3):
        words = words + pad([r[i] for r in reps], cap)
    words = words + pad(row_off, cap) + spill + keep + home_off + first + cnt + pad(spilling, E) + load + rfirst + rcnt
    segs = [(e, e // L, keep[e], (e // L) * C + home_off[e]) for e in range(E)]
    segs += [(e, d, n, d * C + ro) for (e, d, n, _), ro in zip(reps, row_off)]
    return words, segs


def _prepare_expert(case, g, st):
    R, E, S, K, inp, out = (case[k] for k in ("R", "E", "S", "K", "inp", "out"))
    C, dev = S * K, "cuda"
    logits = _normal((R * S, E), g) + case["skew"] * _normal((E,), g)
    counts = torch.bincount(torch.topk(logits, K, dim=1).indices.reshape(-1), minlength=E).tolist()
    words, segs = _plan(R, E, C, counts)
    st["plan"] = torch.tensor(words, dtype=torch.int32, device=dev)
    st["n_rep"] = len(segs) - E
    st["longest"] = max(n for _, _, n, _ in segs)
    st["seg_rows"] = torch.tensor([n for _, _, n, _ in segs], device=dev)
    st["seg_row0"] = torch.tensor([r for _, _, _, r in segs], device=dev)
    st["d_y"] = _bf16((R * C, out), g, 0.1)
    if case["kind"] == "dw":
        st["x"] = _bf16((R * C, inp), g)
        st["home"] = torch.empty((E, out * inp), dtype=torch.float32, device=dev)
        st["replicas"] = torch.zeros((E + R, out * inp), dtype=torch.float32, device=dev)  # rows without a replica stay 0
        st["segs"] = segs
        return
    B = case["B"]
    hosted, wslot = [0] * R, [-1] * (E + R)
    for j, (_, d, _, _) in enumerate(segs[E:]):
        wslot[j] = d * B + hosted[d] if hosted[d] < B else -1
        hosted[d] += 1
    st["wslot"] = torch.tensor(wslot, dtype=torch.int32, device=dev)
    st["w_home"] = _bf16((E, out * inp), g, inp ** -0.5)
    st["pool"] = torch.zeros((R * B, out * inp), dtype=torch.bfloat16, device=dev)
    for j, w in enumerate(wslot):
        if w >= 0:
            st["pool"][w] = st["w_home"][segs[E + j][0]]
    st["seg_weight"] = torch.tensor([e for e in range(E)] + [E + w if w >= 0 else segs[E + j][0]
                                                             for j, w in enumerate(wslot[:st["n_rep"]])], device=dev)
    st["segs"] = segs
    st["d_x"] = torch.empty((R * C, inp), dtype=torch.bfloat16, device=dev)


def _bank(st):
    """A [M, rank, in] and B [M, out, rank] of the bank (or of its gradient)."""
    M, r, inp, out = st["M"], st["rank"], st["inp"], st["out"]
    return lambda b: (b[:, :r * inp].view(M, r, inp), b[:, r * inp:].view(M, out, r))


def _prepare_adapter(case, g, st):
    N, M, r, inp, out = (case[k] for k in ("N", "M", "rank", "inp", "out"))
    dev = "cuda"
    # sequences of random lengths, each with its adapter (M: none)
    cuts = torch.randint(0, N, (case["seqs"],), generator=g, device=dev)
    of_seq = torch.randint(0, M, (case["seqs"] + 1,), generator=g, device=dev)
    of_seq[torch.rand(case["seqs"] + 1, generator=g, device=dev) < case["none"]] = M
    ids = of_seq[torch.cumsum(torch.bincount(cuts, minlength=N), 0)]
    if case["kind"] == "adapter" and case["sorted"]:
        ids = ids[torch.randperm(N, generator=g, device=dev)]
    order = torch.sort(ids, stable=True).indices
    counts = torch.bincount(ids, minlength=M + 1).tolist()
    st["ids"], st["order"] = ids.int(), order.int()
    st["counts"] = torch.tensor(counts, device=dev)
    st["longest"] = max(1, max(counts[:M]))
    st["plan"] = torch.tensor(_plan(1, M + 1, N, counts)[0], dtype=torch.int32, device=dev)
    st["x"] = _bf16((N, inp), g)
    st["bank"] = _bf16((M, r * (inp + out)), g)
    a, b = _bank(st)(st["bank"])
    a *= inp ** -0.5
    b *= 0.3 * r ** -0.5
    st["scale"] = 0.5 + 1.5 * torch.rand(M, generator=g, device=dev)
    if case["kind"] == "adapter":
        st["base"] = _bf16((N, out), g)
        st["y"] = torch.empty_like(st["base"])
        st["u"] = torch.empty((N, r), dtype=torch.float32, device=dev)
        st["workspace"] = torch.empty(64 * N * r + 65536, dtype=torch.uint8, device=dev)
        return
    st["u"] = torch.zeros((N, r), device=dev)
    for m in range(M):
        rows = order[sum(counts[:m]):sum(counts[:m + 1])]
        st["u"][rows] = st["x"][rows].float() @ a[m].float().T
    st["d_y"] = _bf16((N, out), g, 0.1)
    st["base"] = _bf16((N, inp), g, 0.1)
    st["d_x"] = torch.empty_like(st["base"])
    st["d_bank"] = torch.empty((M, r * (inp + out)), dtype=torch.float32, device=dev)
    st["workspace"] = torch.empty(68 * N * r + 4 * (64 + M) * r * (inp + out) + 65536, dtype=torch.uint8, device=dev)


def _prepare_clip(case, g, st):
    """Gradient tensors, one output buffer, and the table of runs: source and
    destination address, elements, type (0 fp32, 1 bf16)."""
    t = torch.bfloat16 if case["bf16"] else torch.float32
    lo, hi = math.log(case["least"]), math.log(case["most"])
    sizes = [int(math.exp(lo + (hi - lo) * (0.618034 * i % 1.0)) + 0.5) for i in range(case["tensors"])]
    if not case["odd"]:
        sizes = [max(8, n - n % 8) for n in sizes]
    st["grads"] = [_normal(n, g, 0.01).to(t) for n in sizes]
    total = sum(sizes)
    st["out"] = torch.empty(total, dtype=t, device="cuda")
    size, at, rows = st["out"].element_size(), 0, []
    for grad, n in zip(st["grads"], sizes):
        src, dst = grad.data_ptr(), st["out"].data_ptr() + at * size
        rows += [(src + i * size, dst + i * size, min(GRAD_RUN, n - i), int(case["bf16"]))
                 for i in range(0, n, GRAD_RUN)]
        at += n
    st["table"] = torch.tensor(rows, dtype=torch.int64).to("cuda")
    st["max_norm"] = 0.01 * math.sqrt(total) / case["ratio"]  # a ratio over 1 clips
    st["norm"] = torch.empty(1, dtype=torch.float32, device="cuda")
    st["workspace"] = torch.empty(65536, dtype=torch.uint8, device="cuda")


def prepare(case, seed):
    st = dict(case)
    make = dict(dx=_prepare_expert, dw=_prepare_expert, adapter=_prepare_adapter, adapter_bwd=_prepare_adapter,
                clip=_prepare_clip)
    make[case["kind"]](case, _gen(seed), st)
    return st


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _padded(st, rows, values):
    """values [rows in segment order, cols] as [segments, longest, cols], zeros
    behind each segment's last row; seg and pos place every row."""
    n = st["seg_rows"]
    seg = torch.repeat_interleave(torch.arange(n.numel(), device=n.device), n, output_size=rows)
    pos = torch.arange(rows, device=n.device) - (torch.cumsum(n, 0) - n)[seg]
    p = torch.zeros((n.numel(), st["longest"], values.shape[1]), device=n.device)
    p[seg, pos] = values
    return p, seg, pos


def _buffer_rows(st, rows):
    """The buffer's rows in segment order."""
    n = st["seg_rows"]
    first = st["seg_row0"] - (torch.cumsum(n, 0) - n)
    return torch.repeat_interleave(first, n, output_size=rows) + torch.arange(rows, device=n.device)


def _plain_dx(st):
    rows = st["d_y"].shape[0]
    at = _buffer_rows(st, rows)
    p, seg, pos = _padded(st, rows, st["d_y"][at].float())
    w = torch.cat([st["w_home"], st["pool"]])[st["seg_weight"]].float().view(-1, st["out"], st["inp"])
    d_x = torch.empty((rows, st["inp"]), device=p.device)
    d_x[at] = torch.bmm(p, w)[seg, pos]
    return dict(d_x=d_x.bfloat16())


def _plain_dw(st):
    rows = st["d_y"].shape[0]
    at = _buffer_rows(st, rows)
    p, _, _ = _padded(st, rows, st["d_y"][at].float())
    q, _, _ = _padded(st, rows, st["x"][at].float())
    d_w = torch.bmm(p.transpose(1, 2), q).view(p.shape[0], -1)
    replicas = torch.zeros_like(st["replicas"])
    replicas[:st["n_rep"]] = d_w[st["E"]:]
    return dict(home=d_w[:st["E"]], replicas=replicas)


def _plain_groups(st):
    """Rows in order of their adapters: their number with an adapter is not read
    back; the rows without one make a group of their own, with zero matrices."""
    order = st["order"].long()
    n = st["counts"]
    group = st["ids"].long()[order]
    pos = torch.arange(order.numel(), device=n.device) - (torch.cumsum(n, 0) - n)[group]
    pos = torch.where(group < st["M"], pos, 0)
    return order, group, pos


def _plain_pad(st, group, pos, values):
    """[M + 1, longest, cols]; what lands in group M is not used."""
    p = torch.zeros((st["M"] + 1, st["longest"], values.shape[1]), device=values.device)
    p[group, pos] = values
    return p[:st["M"]]


def _plain_unpad(st, order, group, pos, p):
    q = torch.cat([p, torch.zeros_like(p[:1])])[group, pos]
    v = torch.empty_like(q)
    v[order] = q
    return v


def _plain_adapter(st):
    a, b = (m.float() for m in _bank(st)(st["bank"]))
    order, group, pos = _plain_groups(st)
    x = _plain_pad(st, group, pos, st["x"][order].float())
    u = torch.bmm(x, a.transpose(1, 2))
    d = torch.bmm(u, b.transpose(1, 2)) * st["scale"][:, None, None]
    y = st["base"].float() + _plain_unpad(st, order, group, pos, d)
    return dict(y=y.bfloat16(), u=_plain_unpad(st, order, group, pos, u))


def _plain_adapter_bwd(st):
    a, b = (m.float() for m in _bank(st)(st["bank"]))
    order, group, pos = _plain_groups(st)
    x = _plain_pad(st, group, pos, st["x"][order].float())
    u = _plain_pad(st, group, pos, st["u"][order])
    d_y = _plain_pad(st, group, pos, st["d_y"][order].float()) * st["scale"][:, None, None]
    d_u = torch.bmm(d_y, b)
    d_x = st["base"].float() + _plain_unpad(st, order, group, pos, torch.bmm(d_u, a))
    d_a = torch.bmm(d_u.transpose(1, 2), x)
    d_b = torch.bmm(d_y.transpose(1, 2), u)
    M = st["M"]
    return dict(d_x=d_x.bfloat16(), d_bank=torch.cat([d_a.view(M, -1), d_b.view(M, -1)], 1))


def _plain_clip(st):
    flat = torch.cat(st["grads"]).float()
    norm = flat.double().square().sum().sqrt()
    factor = torch.clamp(st["max_norm"] / norm, max=1.0).float()
    return dict(norm=norm.float().view(1), out=(flat * factor).to(st["out"].dtype))


_PLAIN = dict(dx=_plain_dx, dw=_plain_dw, adapter=_plain_adapter, adapter_bwd=_plain_adapter_bwd, clip=_plain_clip)


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------

def _own(st):
    import load_balancing_amd as mx

    kind = st["kind"]
    if kind == "clip":
        mx.moonep_grad_clip(st["table"], st["max_norm"], st["norm"], st["workspace"])
        return dict(norm=st["norm"], out=st["out"])
    inp, out = st["inp"], st["out"]
    if kind in ("dx", "dw"):
        s = mx.Shape(st["R"], st["E"], st["S"], st["K"], 8)
        if kind == "dx":
            mx.moonep_expert_gemm_dx(s, st["plan"], st["wslot"], st["B"], inp, out, st["d_y"], st["w_home"],
                                     st["pool"], out * inp, 0, st["d_x"])
            return dict(d_x=st["d_x"])
        mx.moonep_expert_gemm_dw(s, st["plan"], inp, out, st["x"], st["d_y"], False, out * inp, 0, st["home"],
                                 st["replicas"])
        return dict(home=st["home"], replicas=st["replicas"])
    M, r = st["M"], st["rank"]
    s = mx.Shape(1, M + 1, st["N"], 1, 8)
    ad = mx.Adapters(M, r, inp, out, r * (inp + out), 0, r * inp)
    if kind == "adapter":
        mx.moonep_adapter(s, ad, st["ids"], st["order"] if st["sorted"] else None, st["x"], st["bank"],
                          st["scale"], st["base"], st["u"], st["y"], st["workspace"])
        return dict(y=st["y"], u=st["u"])
    mx.moonep_adapter_bwd(s, ad, st["ids"], st["order"], st["plan"], st["x"], st["u"], st["d_y"], st["bank"],
                          st["scale"], st["base"], st["d_x"], False, st["d_bank"], st["workspace"])
    return dict(d_x=st["d_x"], d_bank=st["d_bank"])


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["kind"]](state)


def work(case):
    kind = case["kind"]
    if kind == "clip":
        lo, hi, n = case["least"], case["most"], case["tensors"]
        mean = lo if hi == lo else (hi - lo) / math.log(hi / lo)
        # every gradient read once and written once; reading it again for the norm's factor is the form's own choice
        return dict(bytes=2 * n * mean * (2 if case["bf16"] else 4), flops=3 * n * mean)
    inp, out = case["inp"], case["out"]
    if kind in ("dx", "dw"):
        NK, E = case["R"] * case["S"] * case["K"], case["E"]
        if kind == "dx":
            return dict(bytes=2 * NK * (inp + out) + 2 * min(E, NK) * inp * out, flops=2 * NK * inp * out)
        return dict(bytes=2 * NK * (inp + out) + 4 * E * inp * out, flops=2 * NK * inp * out)
    N, M, r = case["N"], case["M"], case["rank"]
    used = min(M, N, case["seqs"] + 1)
    if kind == "adapter":
        return dict(bytes=N * (2 * inp + 4 * out + 4 * r + 4) + 2 * used * r * (inp + out), flops=2 * N * r * (inp + out))
    return dict(bytes=N * (6 * inp + 2 * out + 4 * r + 8) + (2 * used + 4 * M) * r * (inp + out),
                flops=4 * N * r * (inp + out))


# ---------------------------------------------------------------------------
# the definitions in fp64
# ---------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    kind = case["kind"]
    if kind == "clip":
        total = sum((g.double() ** 2).sum() for g in st["grads"])
        norm = torch.sqrt(total)
        factor = min(1.0, st["max_norm"] / float(norm))
        return dict(norm=norm.view(1), out=torch.cat([g.double() * factor for g in st["grads"]]))
    inp, out = case["inp"], case["out"]
    if kind in ("dx", "dw"):
        E, segs = case["E"], st["segs"]
        if kind == "dx":
            d_x = torch.zeros((st["d_y"].shape[0], inp), dtype=torch.float64, device="cuda")
            for (_, _, n, r0), w in zip(segs, st["seg_weight"].tolist()):
                wm = st["w_home"][w] if w < E else st["pool"][w - E]
                d_x[r0:r0 + n] = st["d_y"][r0:r0 + n].double() @ wm.double().view(out, inp)
            return dict(d_x=d_x)
        g = torch.stack([(st["d_y"][r0:r0 + n].double().T @ st["x"][r0:r0 + n].double()).view(-1)
                         for _, _, n, r0 in segs])
        return dict(home=g[:E], replicas=torch.cat([g[E:], g.new_zeros((2 * E + case["R"] - len(segs), out * inp))]))
    N, M, r = case["N"], case["M"], case["rank"]
    A, B = _bank(st)(st["bank"])
    if kind == "adapter":
        y, u = st["base"].double(), torch.zeros((N, r), dtype=torch.float64, device="cuda")
        for m in range(M):
            at = torch.nonzero(st["ids"] == m)[:, 0]
            u[at] = st["x"][at].double() @ A[m].double().T
            y[at] += st["scale"][m].double() * (u[at] @ B[m].double().T)
        return dict(y=y, u=u)
    d_x, d_bank = st["base"].double(), []
    for m in range(M):
        at = torch.nonzero(st["ids"] == m)[:, 0]
        s = st["scale"][m].double()
        d_y = st["d_y"][at].double()
        d_u = s * (d_y @ B[m].double())
        d_x[at] += d_u @ A[m].double()
        d_a = d_u.T @ st["x"][at].double()
        d_b = s * (d_y.T @ st["u"][at].double())
        d_bank.append(torch.cat([d_a.view(-1), d_b.view(-1)]))
    return dict(d_x=d_x, d_bank=torch.stack(d_bank))
