"""The router's sums over very many tokens."""
import numpy as np
import pytest
import torch

import load_balancing_amd as mx

pytestmark = pytest.mark.gpu


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
