"""The router's scores one by one, and its sums over very many tokens."""
import numpy as np
import pytest
import torch

import load_balancing_amd as mx

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
def test_scores_one_by_one(bf16):
    """Sigmoid's scores are the gates (scale 1, all experts chosen): each within (2.5 |l| + 8) 2^-24 of the true one, or
    below 2^-126 and 0.  Softmax's are the gates of rows of two, (1 + exp(-|x|))^-1 and exp(-|x|) of it: one more
    addition, reciprocal and product, 4 2^-24."""
    rng = np.random.default_rng(51)
    N, E = 4096, 64
    print(f"[case] scores bf16={bf16}", flush=True)
    dev = torch.device("cuda")
    t = torch.from_numpy((rng.random((N, E)) * 200 - 100).astype(np.float32)).to(torch.bfloat16 if bf16 else torch.float32)
    l = t.double().numpy()
    ids, gates = torch.empty(N * E, dtype=torch.int32, device=dev), torch.empty(N * E, device=dev)
    mx.moonep_router(mx.Shape(1, E, N, E, 16), mx.RouterOpts(mx.SCORE_SIGMOID, False, 1, int(bf16)), t.to(dev), ids, gates)
    got = np.empty((N, E))
    np.put_along_axis(got, ids.cpu().numpy().reshape(N, E), gates.double().cpu().numpy().reshape(N, E), 1)
    want = 1 / (1 + np.exp(-l))
    small = want < 2.0 ** -125.9
    assert small.any() and (got[small] < 2.0 ** -125.8).all()
    assert (np.abs(got - want) <= want * (2.5 * np.abs(l) + 8) * 2.0 ** -24)[~small].all()

    two = t.view(N * E // 2, 2)
    l = two.double().numpy()
    n = l.shape[0]
    ids, gates = ids[:2 * n], gates[:2 * n]
    mx.moonep_router(mx.Shape(1, 2, n, 2, 16), mx.RouterOpts(mx.SCORE_SOFTMAX, False, 1, int(bf16)), two.to(dev), ids, gates)
    x = -np.abs(l[:, :1] - l[:, 1:])
    want = np.concatenate([1 / (1 + np.exp(x)), np.exp(x) / (1 + np.exp(x))], 1)
    got = gates.double().cpu().numpy().reshape(n, 2)
    small = want < 2.0 ** -125.9
    assert small.any() and (got[small] < 2.0 ** -125.8).all()
    assert (np.abs(got - want) <= want * (2.5 * np.abs(x) + 12) * 2.0 ** -24)[~small].all()


def test_shares_of_many_tokens():
    """2^24 and more tokens with the same logits, so that every fp32 addition rounds the same way.  A workgroup
    sums at most 2048 tokens in fp32, 128 in a lane and then over 16 lanes: 144 2^-24 at most, beside the share's own
    error (logits up to 1.8 apart: (2 X + 8 + E / 8 + 32) 2^-24) and one rounding of the fp64 sum."""
    N, E, G = (1 << 24) + 4096, 3, 2
    print(f"[case] shares N={N} E={E}", flush=True)
    l = np.array([0.97, -0.06, -0.8], np.float32)
    s, o = mx.Shape(1, E, N, 1, 16), mx.RouterOpts(mx.SCORE_SOFTMAX, False, G)
    d = torch.from_numpy(l).cuda().repeat(N, 1)
    ids, gates = torch.empty(N, dtype=torch.int32, device="cuda"), torch.empty(N, device="cuda")
    counts, prob = torch.empty((G, E), dtype=torch.int32, device="cuda"), torch.empty((G, E), device="cuda")
    loss = torch.empty(1, device="cuda")
    ws = torch.empty(mx.moonep_router_workspace_bytes(s, o), dtype=torch.uint8, device="cuda")
    mx.moonep_router(s, o, d, ids, gates, counts, prob, loss, ws)
    torch.cuda.synchronize()
    v = np.exp(l.astype(np.float64) - np.float64(l[0]))
    p, n = v / v.sum(), N // G
    own = (2 * 1.8 + 8 + E / 8 + 32) * 2.0 ** -24
    assert (counts.cpu().numpy() == [[n, 0, 0]] * G).all() and int(ids.abs().max()) == 0
    np.testing.assert_allclose(prob.cpu().numpy(), [n * p] * G, rtol=own + 145 * 2.0 ** -24)
    # the share as the kernel has it, in the gates: what is left is the summing alone
    np.testing.assert_allclose(prob.cpu().numpy()[:, 0], n * float(gates[0]), rtol=146 * 2.0 ** -24)
    np.testing.assert_allclose(loss.cpu().numpy()[0], E * p[0], rtol=own + 146 * 2.0 ** -24)
