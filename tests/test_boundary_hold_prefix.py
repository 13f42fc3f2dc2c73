"""accept_hold with slots that are not a request's to write, on the host."""
from tests.test_boundary_attn import call
from tests.test_boundary_hold import NAMES
from tests.test_boundary_host import hrs

DESC = dict(n_req=2, n_pos=5, n_pages=8, page_size=16, table_len=4, min_len=0)


def test_min_len():
    for n, want in ((0, hrs.HRS_EDEVICE), (100, hrs.HRS_EDEVICE), (2 ** 31 - 1, hrs.HRS_EDEVICE), (-1, hrs.HRS_EINVAL)):
        assert call("accept_hold", hrs.HoldDesc, NAMES, DESC, dict(min_len=n))[0] == want
