"""The block for a few tokens where the tokens share experts unevenly (marked gpu): an expert of most tokens beside many
of one or none, so that one expert's rows take several readings of its weights.  Values, choices and tolerances as in
test_gpu_forward_few; and each token is the token alone, bit for bit."""
import numpy as np
import pytest
import torch

from routing_dispatch_grouped_router_amd import binding as B
from test_gpu_forward_few import Case

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.mark.parametrize("act", ["f32", "bf16", "mxfp8"])
@pytest.mark.parametrize("padded", [0, 9])
@pytest.mark.parametrize("T, d, E, k, H, share", [(32, 256, 128, 4, 128, 0.7), (32, 128, 64, 8, 192, 1.0), (20, 512, 128, 1, 128, 1.0),
                                                  (32, 128, 8, 4, 64, 1.0), (17, 192, 12, 2, 128, 0.8)])
def test_experts_shared_unevenly(T, d, E, k, H, share, padded, act):
    d, H = (-(-n // 128) * 128 if act == "mxfp8" else n for n in (d, H))
    print(f"[few, skewed] T={T} d={d} E={E} k={k} H={H} {act} padded={padded}", flush=True)
    c = Case(T, d, E, k, H, act, given=True)
    rng = np.random.default_rng(T + E)
    logits = rng.standard_normal((T, E)) - 1.0 * np.log(1 + np.arange(E))       # Zipf's weights
    logits[rng.random(T) < share, E // 2] = 9.0                                 # and one expert of nearly every token
    c.logits = torch.from_numpy(logits.astype(np.float32))
    c.dev["logits"] = c.logits.to(DEV)
    mask = None
    if padded:
        mask = torch.ones(T, dtype=torch.uint8, device=DEV)
        mask[rng.permutation(T)[:padded]] = 0
    c.run(mask=mask)
    c.check(mask)
    want = c.op.y.clone()
    one = B.ForwardFew(B.problem(1, d, E, k, H, act, logits_given=True), DEV)
    for t in range(T):
        if mask is None or mask[t]:
            y = one(c.dev["x"][t:t + 1], c.packed, logits=c.dev["logits"][t:t + 1].contiguous())
            assert torch.equal(y[0], want[t]), t
