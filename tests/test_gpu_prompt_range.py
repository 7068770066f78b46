"""GPU tests of prompt_attention with large rows, up to the documented range: rows a query sees x max|K| < 2^80.

Rows times 2^e and queries times 2^-e have the same logits, to the bit (every product and sum of them has the
same operands but for exact powers of two), so the same probabilities and lse, and results times 2^e, to the bit.
The rows behind the first 128 are alike and have logits above the first ones' by nearly what moves the running
reference, so that the sums come as near to the end of fp32 as they can."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
SM = 512 ** -0.5
LAG = 32 * np.log(2.0)


# e: 2^80 / rows, rounded down, for values of magnitude 1 to 2
@pytest.mark.parametrize("rows,e", [(300, 70), (5000, 66), (20000, 64)])
@pytest.mark.parametrize("n,H", [(1, 5), (3, 128)])
def test_large_rows(gkr, rows, e, n, H):
    assert rows * 2.0 ** (e + 1) < 2.0 ** 80
    rng = np.random.default_rng(rows + H)
    k = rng.choice([-1.0, 1.0], (rows, 512)) * rng.uniform(1, 2, (rows, 512))
    k[128:] = k[128]
    k = torch.from_numpy(k).to(torch.bfloat16)
    kd = k.double().numpy()
    at = 23.0 * rng.uniform(0.99, 1.01, n * H) / (SM * (kd[128] ** 2).sum())
    q = torch.from_numpy(at[:, None] * kd[128]).to(torch.bfloat16)
    s = SM * q.double().numpy() @ kd[:129].T
    above = s[:, 128] - s[:, :128].max(1)
    assert (above < LAG - 0.1).all() and (above > 0.75 * LAG).all()
    starts = torch.arange(n + 1, dtype=torch.int32, device=DEV)
    q, kv = q.view(n, H, 512).to(DEV), torch.cat([k] * n).to(DEV)
    out, lse = gkr.prompt_attention(q, kv, starts, SM, kv_starts=starts * rows)
    assert torch.isfinite(out.float()).all()
    up, down = 2.0 ** e, 2.0 ** -e
    big, big_lse = gkr.prompt_attention(q * down, kv * up, starts, SM, kv_starts=starts * rows)
    assert torch.equal(big_lse, lse) and torch.equal(big, out * up)
