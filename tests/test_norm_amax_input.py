"""The per-tensor norm's amax input is apart from every output.  CPU only: the
host refuses the call."""
import ctypes

import pytest

from test_block_host import G, H, QC, QR, R, RS, X, Y, f  # noqa: F401

vp = ctypes.c_void_p


@pytest.mark.parametrize("place", [RS.value + 16, H.value, Y.value + 512, QR.value + 4, QC.value + 256 * 512 - 4,
                                   0xC000000, 0xD000000])
def test_amax_inside_an_output(f, place):  # noqa: F811
    call = f.lib().fp8_tensor_rmsnorm_quantize
    head = (X, R, G, 256, 512, 512, 512, 1e-6, 0)
    scale, amax_out = vp(0xC000000), vp(0xD000000)
    assert call(*head, vp(place), H, RS, Y, QR, QC, scale, amax_out, None) == f.binding.ERR_INVALID_ARG
