"""Page ids that are none, in the caller's table or free list: they change hands as they are, and the call that
moves one says so (GDN_DEVERR_PAGE), whatever outputs are asked for."""
import numpy as np
import pytest

from gated_deltanet_recurrent_gb300 import abi
from tests.test_gpu_kv_pages import Both, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [-1, 40, 2 ** 31 - 1, -2 ** 31])
def test_given_back_and_handed_out_again(bad):
    b = Both(4, 40, 8, 16)
    b.grow([0, 1, 2], [0, 0, 0], [60, 100, 5])
    b.kv.page_table[1, 2] = bad
    b.ref.table[1, 2] = bad
    b.trim([0, 1], [0, 48])     # the entry stays, and nothing is reported
    abi.gdn_kv_pages_trim(b.kv, b.book, i32([1]), i32([0]))
    assert abi.gdn_kv_get_error(b.kv) == abi.DEVERR_PAGE
    b.ref.trim([1], [0])
    assert b.ref.err
    b.ref.err = 0
    b.same()
    # no outputs: the call reports it all the same
    abi.gdn_kv_pages_grow(b.kv, b.book, i32([3]), i32([0]), i32([0, 128]), 128)
    assert abi.gdn_kv_get_error(b.kv) == abi.DEVERR_PAGE
    b.ref.grow([3], [0], [0, 128], 128, np.zeros(128), np.zeros(128))
    b.ref.err = 0
    b.same()
    b.trim([3], [128])
    b.grow([2], [5], [20])      # others get pages as before


def test_many_pages_in_many_blocks():
    n = 60
    b = Both(n, 20000, 512, 16)
    lens = [8192 - 31 * i for i in range(n)]
    b.grow(range(n), [0] * n, [min(x, 5000) for x in lens])
    b.kv.page_table[n - 1, 200] = 20000
    b.ref.table[n - 1, 200] = 20000
    b.trim(range(n), [17] * n)
    assert b.book.free_pages.tolist().count(20000) == 1
    b.grow(range(n), [17] * n, [4983] * n)


def test_host_checks_refuse_them():
    b = Both(4, 40, 8, 16, host_checks=True)
    b.grow([0, 1], [0, 0], [60, 100])
    b.kv.page_table[1, 2] = -1
    b.ref.table[1, 2] = -1

    def refused(call, *args):
        with pytest.raises(abi.GDNError) as e:
            call(b.kv, b.book, *args)
        assert e.value.name == "GDN_ERR_SIZE"
        b.same()
    refused(abi.gdn_kv_pages_trim, i32([0, 1]), i32([0, 0]))
    b.trim([0, 1], [0, 48])
    top = b.book.n_free.item()
    b.book.free_pages[top - 2] = 40
    b.ref.free[top - 2] = 40
    refused(abi.gdn_kv_pages_grow, i32([2, 3]), i32([0, 0]), i32([0, 5, 10]), 10)
    refused(abi.gdn_kv_pages_grow, i32([2]), i32([0]), i32([0, 17]), 17)
    b.grow([2], [0], [16])
    b.grow([3], [0], [0])


def test_free_pages_that_are_not_reached_may_hold_anything():
    b = Both(2, 6, 3, 16, host_checks=True)
    b.book.free_pages[0] = 77
    b.ref.free[0] = 77
    assert b.grow([0], [0], [48]) == [1]
    assert b.grow([1], [0], [32]) == [1]
