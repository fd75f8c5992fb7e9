"""The routed block on the GPU in rare situations: repeated ids beside infinite weights, infinite norm weights and
gates in rows of every raggedness, slices that start anywhere, and launch variants that need particular sizes.

Bounds as in test_gpu_block.py; where a result is compared with the same call on other inputs, the bits are equal.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU visible", allow_module_level=True)

import swiglu_mlp_fwd_amd as S  # noqa: E402
import test_gpu_block as G  # noqa: E402
from oracle import block_oracle as B  # noqa: E402
from parity_util import check_guards, guarded  # noqa: E402

DEV = G.DEV


# ----------------------------------------------------------------- experts

def repeated_ids(T, E, k, e, full):
    """The first `full` tokens name e in all k entries and the last token once; every other entry names an expert of its
    own, so that what follows e in the order of the entries is other tokens' experts."""
    others = iter([i for i in range(E) if i != e])
    return np.array([[e if t < full or (t == T - 1 and j == 0) else next(others) for j in range(k)] for t in range(T)],
                    np.int32)


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("T,E,k,full,N,K", [
    (8, 60, 8, 1, 72, 4104),     # 9 pairs of one expert, 2 tokens
    (4, 64, 16, 1, 72, 4104),    # 17 pairs, 2 tokens: also more than the 16 columns of the first product
    (16, 64, 4, 2, 72, 4104),    # 9 pairs, 3 tokens
    (32, 64, 2, 8, 136, 4104)])  # 17 pairs, 9 tokens: two passes of tokens in the second product
def test_moe_repeated_ids_of_an_expert_with_non_finite_weights(T, E, k, full, N, K, bad):
    """What the other tokens get does not depend on the weights of an expert that they do not name, however often
    another token names it."""
    e = 3
    x, w = G.normal((T, K), 31, "bf16"), G.normal((T, k), 32, "f32")
    wg, wu = G.normal((E, N, K), 33, "bf16", 0.05), G.normal((E, N, K), 34, "bf16", 0.05)
    wd = G.normal((E, K, N), 35, "bf16", 0.05)
    ids = torch.from_numpy(repeated_ids(T, E, k, e, full)).to(DEV)
    clean = S.moe_fwd(x, wg, wu, wd, ids, w)
    if bad == math.inf:
        want, bound = B.moe_bound(G.host(x), G.host(wg), G.host(wu), G.host(wd), ids.cpu().numpy(), G.host(w), "silu")
        G.within(clean, want, bound, "repeated ids")
    wd[e, ::3] = bad
    y = S.moe_fwd(x, wg, wu, wd, ids, w)
    assert torch.equal(y[full:-1], clean[full:-1])
    named = [*range(full), T - 1]
    assert not torch.isfinite(y[named, ::3]).any()
    keep = torch.arange(K, device=DEV) % 3 != 0
    assert torch.equal(y[:, keep], clean[:, keep])
