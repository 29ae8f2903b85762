"""The training calls on an MI355X over arrays past 4 GiB and windows past 2^32
bytes of a row, with integers whose sums are exact: compared bit for bit."""
import pytest
import torch

import load_balancing_amd as mx

pytestmark = pytest.mark.gpu

FAR = (1 << 31) + 8  # elements


def ints(shape):
    return torch.randint(-1, 2, shape, device="cuda", dtype=torch.int8).bfloat16()


def layer(rows):
    s = mx.Shape(1, 2, rows, 1, 8)
    b = mx.allocate(s)
    mx.plan_step(b, torch.randint(0, 2, (rows,), device="cuda").int())
    return s, b


def segments(b):
    f = b.plan_fields()
    return [(int(f["home_row_off"][e]), int(f["keep"][e]), e) for e in range(2)]


def test_rows_past_4_gib(gpu_ready):
    rows, inp, out = 540000, 4096, 128  # x and d_x: 4.4e9 bytes
    s, b = layer(rows)
    x, dy, w = ints((rows, inp)), ints((rows, out)), ints((2, out * inp))
    dx = torch.empty_like(x)
    wslot = torch.full((3,), -1, dtype=torch.int32, device="cuda")
    mx.moonep_expert_gemm_dx(s, b.plan, wslot, 0, inp, out, dy, w, None, out * inp, 0, dx)
    home, rep = torch.empty((2, out * inp), device="cuda"), torch.empty((3, out * inp), device="cuda")
    mx.moonep_expert_gemm_dw(s, b.plan, inp, out, x, dy, False, out * inp, 0, home, rep)
    for r0, n, e in segments(b):
        want = torch.zeros((out, inp), device="cuda")
        for at in range(r0, r0 + n, 1 << 16):
            end = min(at + (1 << 16), r0 + n)
            d = dy[at:end].float()
            # at most 128 and 540000 ones: exact in bf16 and in fp32
            assert torch.equal(dx[at:end], (d @ w[e].float().view(out, inp)).bfloat16())
            want += d.T @ x[at:end].float()
        assert torch.equal(home[e].view(out, inp), want)


def test_windows_past_4_gib(gpu_ready):
    """Weights and gradients whose window begins behind 2^31 elements of a row of their bank."""
    rows, inp, out = 700, 64, 128
    s, b = layer(rows)
    n, stride = out * inp, FAR + out * inp
    x, dy = ints((rows, inp)), ints((rows, out))
    bank = torch.empty((2, stride), dtype=torch.bfloat16, device="cuda")
    w = bank[:, FAR:]
    w.copy_(ints((2, n)))
    dx = torch.empty_like(x)
    wslot = torch.full((3,), -1, dtype=torch.int32, device="cuda")
    mx.moonep_expert_gemm_dx(s, b.plan, wslot, 0, inp, out, dy, bank, None, stride, FAR, dx)
    home = torch.empty((2, stride), device="cuda")
    rep = torch.empty((3, stride), device="cuda")
    mx.moonep_expert_gemm_dw(s, b.plan, inp, out, x, dy, False, stride, FAR, home, rep)
    for r0, k, e in segments(b):
        d = dy[r0:r0 + k].float()
        assert torch.equal(dx[r0:r0 + k], (d @ w[e].float().view(out, inp)).bfloat16())
        assert torch.equal(home[e, FAR:].view(out, inp), d.T @ x[r0:r0 + k].float())


@pytest.mark.parametrize("N,inp,out,gap", [(270000, 8200, 8, 0), (270000, 8, 8200, 0), (300, 64, 72, FAR),
                                           (20, 64, 72, FAR)])
def test_adapters_past_4_gib(gpu_ready, N, inp, out, gap):
    M, rank = 2, 8
    s = mx.Shape(1, M + 1, N, 1, 8)
    stride = gap + rank * (inp + out)
    ad = mx.Adapters(M, rank, inp, out, stride, gap, gap + rank * inp)
    ids = torch.randint(0, M + 1, (N,), device="cuda").int()
    b = mx.allocate(s)
    mx.plan_step(b, ids)
    x, base, dy, dx_base = ints((N, inp)), ints((N, out)), ints((N, out)), ints((N, inp))
    x[:, :-8] = 0   # u, du at most 8, sums over rows at most 8 N: exact
    dy[:, :-8] = 0
    bank = torch.empty((M, stride), dtype=torch.bfloat16, device="cuda")
    d_bank = torch.empty((M, stride), device="cuda")
    mats = lambda t, m: (t[m, gap:gap + rank * inp].view(rank, inp), t[m, gap + rank * inp:].view(out, rank))  # noqa: E731
    for m in range(M):
        for t in mats(bank, m):
            t.copy_(ints(t.shape))
    scale = torch.ones(M, device="cuda")
    y, u, dx = torch.empty_like(base), torch.empty((N, rank), device="cuda"), torch.empty_like(dx_base)
    work = torch.empty(max(mx.moonep_adapter_workspace_bytes(s, ad), mx.moonep_adapter_bwd_workspace_bytes(s, ad)),
                       dtype=torch.uint8, device="cuda")
    mx.moonep_adapter(s, ad, ids, b.src_of_slot, x, bank, scale, base, u, y, work)
    mx.moonep_adapter_bwd(s, ad, ids, b.src_of_slot, b.plan, x, u, dy, bank, scale, dx_base, dx, False, d_bank, work)
    sums = [[torch.zeros(t.shape, device="cuda") for t in mats(bank, m)] for m in range(M)]
    for at in range(0, N, 1 << 15):
        part = slice(at, at + (1 << 15))
        i, X, D, Y, U, DX = ids[part], x[part].float(), dy[part].float(), base[part].float(), u[part], dx_base[part].float()
        for m in range(M):
            A, B = (t.float() for t in mats(bank, m))
            mine = (i == m).float()[:, None]
            uu, du = X @ A.T * mine, D @ B * mine
            assert torch.equal(U * mine, uu)
            Y += uu @ B.T
            DX += du @ A
            sums[m][0] += du.T @ X
            sums[m][1] += D.T @ uu
        assert torch.equal(y[part], Y.bfloat16()) and torch.equal(dx[part], DX.bfloat16())
    for m in range(M):
        for got, want in zip(mats(d_bank, m), sums[m]):
            assert torch.equal(got, want)


def test_clip_past_2_31_elements(gpu_ready):
    n = FAR + 3
    g = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    g[-1] = 1.0 + 2.0 ** -7
    h = torch.full((5,), 2.0, device="cuda")
    table = mx.moonep_grad_table([g, h])
    norm, work = torch.empty(1, device="cuda"), torch.empty(mx.GRAD_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    total = (n - 1 + (1.0 + 2.0 ** -7) ** 2 + 20.0) ** 0.5
    mx.moonep_grad_clip(table, total / 4, norm, work)
    assert abs(norm.item() - total) <= 2.0 ** -23 * total
    # factors of 1/4 but for the roundings of fp32: bf16 rounds them away
    assert (g[:-1] == 0.25).all() and g[-1].item() == (1.0 + 2.0 ** -7) / 4
    assert ((h - 0.5).abs() <= 2.0 ** -23).all()
