"""Calls of more work than the kernels can count are refused on the host, before anything is enqueued (and before a
device is looked for: no GPU needed)."""
import torch

from lora_moe_gb300 import binding as B
from test_fp8_arguments import P0, UNSUPPORTED, _dense, _grouped, _naive

NO_DEVICE = 6     # what a valid call returns here


def _valid(status):
    """A call with valid arguments goes on to the device: it is not tried where there is one, as its pointers are not."""
    return status == NO_DEVICE


def test_too_many_items():
    n = 1 << 30
    assert _dense(M=1 << 29, N=n, ldy=n) == UNSUPPORTED                        # 2^21 x 2^22 tiles of 256 x 256
    assert _grouped(M=1 << 28, N=n, ldy=n, cap=(1 << 29) + 8 * 15, capb=1 << 26) == UNSUPPORTED
    big = 1 << 29                                                              # 2^24 pairs by 2^22 tiles of 128 columns
    assert _naive(M=1 << 23, N=big, ldy=big) == UNSUPPORTED


def test_the_largest_that_fit():
    if torch.cuda.is_available():
        return
    n = 1 << 23
    assert _valid(_dense(M=1 << 19, N=n, ldy=n))            # 2^11 x 2^15 = 2^26 tiles, of 2^27 - 1
    assert _valid(_dense(M=64, N=1 << 30, ldy=1 << 30))     # few rows: 4 x 2^23 items
    m = 1 << 18                                             # 2^11 + 8 tiles
    need = B.fp8_grouped_workspace_bytes(m, 2, 8, 256, n, 16)
    assert need > 0
    assert _valid(_grouped(M=m, N=n, ldy=n, cap=(m * 2) + 8 * 15, capb=1 << 26, ws_ptr=P0, ws_bytes=need))
    assert _valid(_naive(M=1 << 8, N=n, ldy=n))
