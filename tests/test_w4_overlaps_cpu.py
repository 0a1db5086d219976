"""Storing a matrix into its own memory, or reading one back over its codes, is refused: kernels would read what they wrote."""
import pytest
import torch

from test_w4_cpu import B, PTR, weight   # noqa: F401  (B is a fixture)

FAR = PTR + (1 << 20)
BYTES, ROW = 64 * 128, 256                       # of the codes; columns of a row


def both(B, src, stride=ROW, dtype=0, **kw):   # noqa: F811
    w = weight(B, **dict(dict(codes=FAR, scales=FAR + (1 << 18)), **kw))
    lib = B.lib()
    return lib.dec_w4_quantize(w, src, stride, dtype, None), lib.dec_w4_dequantize(w, src, stride, dtype, None)


@pytest.mark.parametrize("src, stride, dtype", [(FAR, ROW, 0), (FAR, ROW, 1), (FAR - 64 * ROW * 4 + 16, ROW, 0), (FAR + BYTES - 16, ROW, 0),
                                                (FAR + (1 << 18) + 256, ROW, 1), (FAR + (1 << 18) - 64 * ROW * 2 + 16, ROW, 1),
                                                (FAR - 5 * 4096 * 4, 4096, 0), (FAR - 5 * 4096 * 4 - ROW * 4 + 16, 4096, 0),
                                                (FAR - 5 * 4096 * 4 + 4096, 4096, 0)])
def test_refused(B, src, stride, dtype):   # noqa: F811
    for rc in both(B, src, stride, dtype):
        assert rc == 1 and "overlap" in B.last_error(None)


def test_codes_and_scales_of_a_store(B):   # noqa: F811
    assert both(B, PTR, scales=FAR + BYTES - 2)[0] == 1 and "overlap" in B.last_error(None)
    assert both(B, PTR, scales=FAR - 62)[0] == 1


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are made up: only for where no kernel can run")
@pytest.mark.parametrize("src, stride, dtype", [(PTR, ROW, 0), (FAR - 64 * ROW * 4, ROW, 0), (FAR + BYTES, ROW, 0), (FAR - 64 * ROW * 2, ROW, 1),
                                                # the codes, and the scales, between two rows of a wider matrix
                                                (FAR - 4096 * 4 - ROW * 4, 4096, 0), (FAR + (1 << 18) - 4096 - ROW * 2, 2048, 1)])
def test_side_by_side(B, src, stride, dtype):   # noqa: F811
    assert both(B, src, stride, dtype) == (5, 5), B.last_error(None)
