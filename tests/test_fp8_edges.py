"""The block-128 quantizer of the oracle next to zero.  CPU only."""
import numpy as np

from oracle import fp8 as ofp8


def test_blocks_whose_scale_has_no_float32_value():
    """amax / 448 rounds to 0 up to half the smallest subnormal (the tie included): the scale is 1, the codes zeros with their signs."""
    step = 2.0 ** -149
    x = np.zeros((4, 128), np.float32)
    x[0, :2], x[1, :2], x[2, :2] = (-224 * step, step), (225 * step, -step), (448 * step, -100 * step)
    codes, scale = ofp8.quantize_block128(x)
    assert scale[:, 0].tolist() == [1.0, step, step, 1.0]
    # 225 steps are 224 to three bits of mantissa, 100 are 96 or 104 (a tie: the even one)
    assert codes[0, :2].tolist() == [0x80, 0] and ofp8.decode_e4m3(codes[1, :2]).tolist() == [224, -1]
    assert ofp8.decode_e4m3(codes[2, :2]).tolist() == [448, -96] and (codes[:, 2:] == 0).all()
