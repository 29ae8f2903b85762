"""The router's sums over very many tokens."""
import numpy as np
import pytest
import torch

import load_balancing_amd as mx

pytestmark = pytest.mark.gpu


def test_shares_of_many_tokens():
    """2^24 and more tokens with the same logits, so that every fp32 addition rounds the same way.  A workgroup
    sums at most 1024 tokens in fp32, 64 in a lane and then 16 lanes: 80 2^-24 at most, beside the share's own 2^-20
    (logits up to 2: (2 X + 8 + E / 8 + 32) 2^-24) and one rounding of the fp64 sum."""
    N, E, G = (1 << 24) + 4096, 3, 2
    print(f"[case] shares N={N} E={E}", flush=True)
    l = np.array([0.7, -1.3, 0.2], np.float32)
    s, o = mx.Shape(1, E, N, 1, 16), mx.RouterOpts(mx.SCORE_SOFTMAX, False, G)
    d = torch.from_numpy(l).cuda().repeat(N, 1)
    ids, gates = torch.empty(N, dtype=torch.int32, device="cuda"), torch.empty(N, device="cuda")
    counts, prob = torch.empty((G, E), dtype=torch.int32, device="cuda"), torch.empty((G, E), device="cuda")
    loss = torch.empty(1, device="cuda")
    ws = torch.empty(mx.moonep_router_workspace_bytes(s, o), dtype=torch.uint8, device="cuda")
    mx.moonep_router(s, o, d, ids, gates, counts, prob, loss, ws)
    torch.cuda.synchronize()
    v = np.exp(l.astype(np.float64) - 0.7)
    p, n = v / v.sum(), N // G
    own = (2 * 2 + 8 + E / 8 + 32) * 2.0 ** -24
    assert (counts.cpu().numpy() == [[n, 0, 0]] * G).all() and int(ids.abs().max()) == 0
    np.testing.assert_allclose(prob.cpu().numpy(), [n * p] * G, rtol=own + 81 * 2.0 ** -24)
    # the share as the kernel has it, in the gates: what is left is the summing alone
    np.testing.assert_allclose(prob.cpu().numpy()[:, 0], n * float(gates[0]), rtol=82 * 2.0 ** -24)
    np.testing.assert_allclose(loss.cpu().numpy()[0], E * p[0], rtol=own + 82 * 2.0 ** -24)
