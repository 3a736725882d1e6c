"""Index arrays that are not aligned to their 4 bytes are refused at the C entries of the page calls."""
import pytest

from gated_deltanet_recurrent_gb300 import abi
from tests.test_gpu_kv_pages import Both, i32

pytestmark = pytest.mark.gpu


def test_nothing_is_launched():
    b = Both(3, 12, 4, 16)
    slots, pos, cu = i32([0, 1]), i32([0, 0]), i32([0, 5, 9])
    lib, book = abi.load_library(), b.book.desc_ptr
    at = [t.data_ptr() for t in (slots, pos, cu)]
    for which in range(3):
        p = [x + 2 * (i == which) for i, x in enumerate(at)]
        st = lib.gdn_kv_pages_grow(b.kv.handle, book, *p, 2, 9, None, None, None, None)
        assert abi.STATUS[st] == "GDN_ERR_ARG"
        if which < 2:
            st = lib.gdn_kv_pages_trim(b.kv.handle, book, p[0], p[1], 2, None)
            assert abi.STATUS[st] == "GDN_ERR_ARG"
    b.same()
    b.grow([0, 1], [0, 0], [5, 4])
