"""The bounded waits of gdn_kv_attend, made to run out without a fault: the
test hook GDN_TEST_KV_WAIT_TIMEOUT gives every other CTA a barrier that waits
for more than it gets.  Such a CTA reports GDN_DEVERR_TIMEOUT; the rows that it
had a part in keep what o held (the workspace holds an earlier call's sums,
which must not come out instead), all others are right, and with the hook
cleared the same call is right again."""
import numpy as np
import pytest
import torch

from gated_deltanet_recurrent_gb300 import abi
from tests.gpu_util import dev, dev_i32
from tests.test_gpu_kv_attend import assert_close, filled, queries
from tests.test_gpu_kv_cache import cum

pytestmark = pytest.mark.gpu


def attend(kv, slots, kv_lens, n, q, max_kv_len):
    o = torch.full(q.shape, 7.0, device="cuda")
    lens = [n] * len(slots)
    abi.gdn_kv_attend(kv, 0, dev_i32(slots), dev_i32(kv_lens), q, o,
                      cu_seqlens=None if n == 1 else cum(lens), max_seqlen=n,
                      max_kv_len=max_kv_len, scale=0.1)
    return o


@pytest.mark.parametrize("h_q,h_kv,d,n", [(8, 2, 128, 1), (16, 2, 256, 1), (8, 2, 128, 6),
                                          (8, 2, 128, 20), (8, 2, 128, 40), (8, 2, 128, 80),
                                          (16, 2, 256, 12), (16, 2, 256, 40), (12, 4, 64, 40)])
def test_a_context_that_is_cut(h_q, h_kv, d, n):
    """Every row has parts in several CTAs (n = 1, 6: the split kernel; else the
    tensor-core kernel, alone and in pairs), so every row is missing."""
    rng = np.random.default_rng(n)
    kv, ref = filled(rng, "i8", 64, h_q, h_kv, d, [3000, 2900])
    q = queries(rng, n, h_q, d, "bf16")
    qd = dev(q, "bf16")
    hint = 8000 if n > 6 else 3000
    attend(kv, [1], [2900], n, qd, hint)               # leaves sums in the workspace
    abi.gdn_kv_set_test_flags(kv, abi.TEST_KV_WAIT_TIMEOUT)
    o = attend(kv, [0], [3000], n, qd, hint)
    assert abi.gdn_kv_get_error(kv) == abi.DEVERR_TIMEOUT
    assert (o == 7).all()
    abi.gdn_kv_set_test_flags(kv, 0)
    o = attend(kv, [0], [3000], n, qd, hint)
    want, mag = ref.attend(0, [0], [3000], [n], q, 0.1)
    assert_close(o, want, mag, "bf16", "f32")
    assert abi.gdn_kv_get_error(kv) == 0


@pytest.mark.parametrize("h_q,h_kv,d,n,n_seqs", [(8, 1, 128, 1, 100), (8, 1, 128, 20, 100),
                                                 (8, 1, 128, 30, 100), (8, 1, 256, 30, 60),
                                                 (8, 1, 128, 80, 60)])
def test_contexts_of_one_cta_each(h_q, h_kv, d, n, n_seqs):
    """Every sequence is one CTA's (or one pair's) whole work: about half of
    them are missing, the others are right."""
    rng = np.random.default_rng(n + 1)
    kv, ref = filled(rng, "e4m3", 64, h_q, h_kv, d, [64, 60, 63])
    slots = [i % 3 for i in range(n_seqs)]
    kv_lens = [[64, 60, 63][s] for s in slots]
    n = min(n, 60)
    q = queries(rng, n * n_seqs, h_q, d, "bf16")
    qd = dev(q, "bf16")
    hint = 64 if n == 1 else 200000
    good = attend(kv, slots, kv_lens, n, qd, hint)
    abi.gdn_kv_set_test_flags(kv, abi.TEST_KV_WAIT_TIMEOUT)
    o = attend(kv, slots, kv_lens, n, qd, hint)
    assert abi.gdn_kv_get_error(kv) == abi.DEVERR_TIMEOUT
    abi.gdn_kv_set_test_flags(kv, 0)
    gone = (o == 7).flatten(1).all(1).view(n_seqs, n)
    assert (gone.all(1) | (~gone).all(1)).all()
    lost = int(gone.all(1).sum())
    assert n_seqs // 3 <= lost <= n_seqs - n_seqs // 3
    keep = ~gone.flatten()
    assert torch.equal(o[keep], good[keep])
    want, mag = ref.attend(0, slots, kv_lens, [n] * n_seqs, q, 0.1)
    assert_close(attend(kv, slots, kv_lens, n, qd, hint), want, mag, "bf16", "f32")
    with pytest.raises(abi.GDNError) as e:
        abi.gdn_kv_set_test_flags(kv, 2)
    assert e.value.name == "GDN_ERR_ARG"
