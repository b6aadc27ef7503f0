"""The bounded waits of the 8-bit product: one warp of a tile gives up where the others do not.

The test build of the library can have the first warp of a tile's sums take its first wait as run out
(gdn_debug_set_matmul_give_up); the others' waits succeed, or end after a short limit where they wait for that warp.  The
kernel has to end, report GDN_ERR_TIMEOUT and leave the next call clean."""
from __future__ import annotations

import pytest
import torch

from tests.fp8_reference import DEV, assert_within, codes_of, product
from tests.gpu_common import lib

pytestmark = pytest.mark.gpu
GDN_ERR_TIMEOUT = 5


# small tiles with rows of any alignment and of whole sectors, alone and with k shared; large tiles alone, several to a CTA, shared:
# with as many blocks as results fit in tensor memory, so that no other warp waits for the one that left, and with more
@pytest.mark.parametrize("T,N,K", [(128, 9727, 640), (128, 9727, 2560), (128, 9728, 640), (40, 700, 600), (40, 700, 5000),
                                   (300, 9001, 256), (300, 9001, 640), (2500, 4099, 640), (128, 10240, 5120)])
def test_one_warp_gives_up(T, N, K):
    g = lib()
    gen = torch.Generator(device=DEV).manual_seed(T + N + K)
    x, xs = codes_of(gen, T, K, 1)
    w, ws = codes_of(gen, N, K, 128)
    out = torch.empty(T, N, dtype=torch.bfloat16, device=DEV)
    with g.using_test_library():
        g.gdn_check_device_errors()  # starts clean
        g.gdn_debug_set_matmul_give_up(True)
        try:
            g.gdn_fp8_matmul(x, xs, w, ws, out=out)
            with pytest.raises(g.GdnError) as e:
                g.gdn_check_device_errors()
            assert e.value.status == GDN_ERR_TIMEOUT
        finally:
            g.gdn_debug_set_matmul_give_up(False)
        g.gdn_fp8_matmul(x, xs, w, ws, out=out)
        g.gdn_check_device_errors()
    want, tol = product(x, xs, w, ws, torch.bfloat16)
    assert_within(out, want, tol, "the next call")
