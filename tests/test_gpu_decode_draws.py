"""The tokens that the decode loop draws, against a 64-bit sampler on the step's own logits and random numbers."""
import numpy as np
import pytest
import torch

from test_gpu_decode_example import SMALL
from test_gpu_decode_ops import sample64

pytestmark = pytest.mark.gpu


def drawn64(row, u, p, mp):
    order, e = sample64(row, 0.8, 50, p, mp)
    up = np.cumsum(e)
    return int(order[min(int((up <= u * up[-1]).sum()), len(order) - 1)])


def test_the_loop_draws_what_its_logits_and_random_numbers_give():
    """float32 exponentials and masses are within 1e-5: a draw is compared where a shift of u and of the filters' edges
    by 1e-4 either way leaves its token the same."""
    import decode
    m = decode.Decoder(5, **SMALL)
    assert [float(m.sampling[k][0]) for k in ("temperature", "top_k", "top_p", "min_p")] == pytest.approx([0.8, 50, 0.95, 0.02])
    steps = []
    step = m.step

    def recorded():
        u = m.u.clone()
        step()
        steps.append((u, m.logits.clone()))
    m.step = recorded
    drawn = m.generate(torch.arange(5, device="cuda"), 32, seed=9, graph=False)
    compared, others = 0, 0
    for i, (u, logits) in enumerate(steps):
        for b in range(5):
            x, at = logits[b], float(u[b])
            want = {drawn64(x, at + du, 0.95 + dp, 0.02 + dm) for du in (-1e-4, 0.0, 1e-4) for dp in (-1e-4, 0.0, 1e-4) for dm in (-2e-6, 0.0, 2e-6)}
            if len(want) == 1:
                compared += 1
                assert int(drawn[i, b]) == want.pop()
                others += int(drawn[i, b]) != int(x.argmax())
    assert compared >= 120 and others >= 40                              # of 160, not the largest logit's alone
