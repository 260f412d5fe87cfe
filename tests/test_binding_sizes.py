"""Sizes that a C int cannot hold are refused by the binding: passed on, they
would be cut to 32 bits and name another, smaller product.  On meta tensors,
which have a shape and no memory; the library is never called."""
import pytest

import gemv_fp16_amd as gf

torch = pytest.importorskip("torch")

BIG = 2 ** 32 + 8


@pytest.fixture(autouse=True)
def _no_library(monkeypatch):
    monkeypatch.setattr(gf, "_ptr", lambda t, dtype, name: 0x10000)

    def launch(name, tensors, stream, *args):
        raise AssertionError("%s reached with %s" % (name, args))

    monkeypatch.setattr(gf, "_launch", launch)


def _meta(*shape, dtype=torch.float16):
    return torch.empty(shape, dtype=dtype, device="meta")


def _off(E):
    return _meta(E + 1, dtype=torch.int32)


def _weights(*lead, K):
    return (_meta(*lead, K // 8, dtype=torch.int32), _meta(*lead, (K + 31) // 32),
            _meta(*lead, (K + 31) // 32, dtype=torch.uint8))


CALLS = {
    "grouped nt, rows": lambda: gf.gemm_f16_grouped_nt(_meta(BIG, 8), _meta(2, 16, 8), _off(2)),
    "grouped nt, columns": lambda: gf.gemm_f16_grouped_nt(_meta(4, 8), _meta(2, BIG, 8), _off(2)),
    "grouped nt, contraction": lambda: gf.gemm_f16_grouped_nt(_meta(4, BIG), _meta(2, 16, BIG), _off(2)),
    "grouped nt, groups": lambda: gf.gemm_f16_grouped_nt(_meta(4, 8), _meta(BIG, 16, 8), _off(BIG)),
    "grouped nn, rows": lambda: gf.gemm_f16_grouped_nn(_meta(BIG, 8), _meta(2, 8, 16), _off(2)),
    "grouped nn, columns": lambda: gf.gemm_f16_grouped_nn(_meta(4, 8), _meta(2, 8, BIG), _off(2)),
    "grouped tn, rows": lambda: gf.gemm_f16_grouped_tn(_meta(BIG, 8), _meta(BIG, 16), _off(2)),
    "grouped tn, columns": lambda: gf.gemm_f16_grouped_tn(_meta(4, 8), _meta(4, BIG), _off(2)),
    "quantize, rows": lambda: gf.w4_quantize_f16(_meta(BIG, 8), 32),
    "quantize, rows of several weights": lambda: gf.w4_quantize_f16(_meta(4, 2 ** 30 + 2, 8), 32),
    "dequantize, rows of several weights": lambda: gf.w4_dequantize_f16(*_weights(4, 2 ** 30 + 2, K=8), 32),
    "quantize, K": lambda: gf.w4_quantize_f16(_meta(4, BIG), 32),
    "dequantize, rows": lambda: gf.w4_dequantize_f16(*_weights(BIG, K=8), 32),
    "dequantize, K": lambda: gf.w4_dequantize_f16(*_weights(4, K=BIG), 32),
    "w4, rows": lambda: gf.gemm_w4_f16_nt(_meta(BIG, 8), *_weights(16, K=8), group=32),
    "w4, columns": lambda: gf.gemm_w4_f16_nt(_meta(4, 8), *_weights(BIG, K=8), group=32),
    "w4, contraction": lambda: gf.gemm_w4_f16_nt(_meta(4, BIG), *_weights(16, K=BIG), group=32),
    "gemv w4, rows": lambda: gf.gemv_w4_f16(*_weights(BIG, K=8), _meta(8), group=32),
    "w4 grouped, rows": lambda: gf.gemm_w4_f16_grouped_nt(_meta(BIG, 8), *_weights(2, 16, K=8), _off(2), group=32),
    "w4 grouped, columns": lambda: gf.gemm_w4_f16_grouped_nt(_meta(4, 8), *_weights(2, BIG, K=8), _off(2), group=32),
}


@pytest.mark.parametrize("name", CALLS)
def test_sizes_past_a_c_int_are_refused(name):
    with pytest.raises(ValueError, match="2\\^31"):
        CALLS[name]()


def test_sizes_at_the_limit():
    gf._ints(2 ** 31 - 1)
    with pytest.raises(ValueError):
        gf._ints(2 ** 31)


def test_sizes_of_a_c_int_reach_the_library():
    with pytest.raises(AssertionError, match="reached"):
        gf.w4_quantize_f16(_meta(2 ** 31 - 1, 8), 32)
