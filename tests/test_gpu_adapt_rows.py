"""Single rows of any width: one output, one token, one adapter of rank 1."""
import numpy as np
import pytest
import torch

from gated_deltanet_recurrent_gb300 import abi
from oracle.adapt_oracle import adapted

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [1, 2, 70, 2100])
@pytest.mark.parametrize("hidden", [100, 3, 8, 257])
@pytest.mark.parametrize("n_out,n,rank", [(1, 1, 1), (1, 3, 8), (16, 1, 1), (1, 1, 5)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_single_rows(tokens, hidden, n_out, n, rank, dtype):
    rng = np.random.default_rng(hidden)
    whole = lambda *s: rng.integers(-2, 3, s).astype(np.float64)
    x, w, a, b = whole(tokens, hidden), whole(n_out, hidden), whole(n, rank, hidden), whole(n, n_out, rank)

    def rows(v):
        """Packed where there is one row, else with a stride of a multiple of 8."""
        t = torch.from_numpy(v).float().cuda().bfloat16()
        if t.numel() == t.shape[-1]:
            return t
        wide = torch.full((*t.shape[:-1], -(-t.shape[-1] // 8) * 8), float("nan"), device="cuda").bfloat16()
        wide[..., :t.shape[-1]] = t
        return wide[..., :t.shape[-1]]
    ids = np.arange(tokens) % (n + 1) - 1
    store = torch.full((tokens, -(-n_out // 8) * 8), 77.0, dtype=dtype, device="cuda")
    y = store[:, :n_out]
    pool = abi.Pool(1, 1, 1, 1, 16, 16, 48, 4, host_checks=False)
    abi.gdn_in_proj_adapted(pool, abi.Adapters(rows(a), rows(b)), rows(x), rows(w),
                            torch.tensor(ids, dtype=torch.int32, device="cuda"), y)
    want = torch.from_numpy(adapted(x, w, a, b, np.ones(n), ids)[0]).to(dtype)
    assert torch.equal(y.cpu(), want)
    assert (store[:, n_out:] == 77).all() and abi.gdn_pool_get_error(pool) == 0
    pool.close()
