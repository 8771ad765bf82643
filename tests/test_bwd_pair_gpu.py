"""The head_dim-256 backward gives the same dK and dV in every run."""
import pytest
import torch

import exact_attention_129_b200 as ea

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("causal", [False, True])
def test_key_gradients_repeat(causal):
    # one query head per key head: dK and dV are sums in a fixed order.  Four segments of
    # 8192 keep the clusters of two CTAs far enough apart that a product which did not
    # wait for its rows to land showed in about one run of twenty
    t, h, d, n = 32768, 8, 256, 80
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v, do = (torch.randn(t, h, d, generator=g, device="cuda").to(torch.bfloat16)
                   for _ in range(4))
    cu = torch.arange(0, t + 1, t // 4, dtype=torch.int32, device="cuda")
    out, lse = ea.attn_fwd(q, k, v, cu, cu, t // 4, t // 4, causal=causal)
    first, differ = None, torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(n):
        _, dk, dv = ea.attn_bwd(q, k, v, out, lse, do, cu, cu, t // 4, t // 4, causal=causal)
        first = first or (dk, dv)
        for a, b in zip((dk, dv), first):
            differ += (a.view(torch.int16) != b.view(torch.int16)).sum()
    rc, msg = ea.last_device_error()
    assert rc == 0, msg
    assert int(differ) == 0
