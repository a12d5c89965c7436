"""The 8-bit base over the whole range of bf16: tokens and weights whose sizes
are far apart, where the product is an ordinary number.

The bound is that of a product alone: four float32 roundings of the value, then
one to bf16."""

import numpy as np
import pytest

from _helpers import bf16_f64, to_dev, to_host_bits
from bit_nf4_quantized_19_amd import synth
from oracle import int8 as oi8

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

U8, U24 = 2.0 ** -8, 2.0 ** -24


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from bit_nf4_quantized_19_amd import ops as o
    o.lib()
    return o


def power(bits, e):
    """bf16 bits times 2^e, by the exponent (values stay normal)."""
    b = bits.astype(np.int32)
    return np.where(b & 0x7FFF, b + (e << 7), b).astype(np.uint16)


@pytest.mark.parametrize("M", [1, 5, 16, 40, 300])
@pytest.mark.parametrize("ex,ew", [(0, 0), (118, -110), (100, -100), (97, -20), (-100, 110),
                                   (-112, 118), (118, 118), (-110, -30)])
def test_tokens_and_weights_of_far_sizes(ops, M, ex, ew):
    print(f"[int8 range] M={M} 2^{ex} 2^{ew}", flush=True)
    d, k = 136, 320
    unit = lambda shape, seed: np.clip(bf16_f64(synth.normal_bf16(shape, 1.0, seed)), -4, 4)  # noqa: E731
    as_bits = lambda v: to_host_bits(torch.from_numpy(v).bfloat16())                          # noqa: E731
    x, wv = unit((M, k), 1 + M), unit((d, k), 2)
    # neither normal's small values leave bf16's normal range
    x, wv = np.where(abs(x) < 2 ** -7, 0, x), np.where(abs(wv) < 2 ** -7, 0, wv)
    X, W = power(as_bits(x), ex), power(as_bits(wv), ew)
    w = ops.quantize_int8(to_dev(W))
    Y, _ = ops.linear_fwd_int8(w, to_dev(X))
    codes, scale = oi8.record(bf16_f64(W).astype(np.float32))
    want, _ = oi8.forward(codes, scale, bf16_f64(X).astype(np.float32))
    got = bf16_f64(to_host_bits(Y))
    if ex + ew > 130:   # past bf16's largest: infinities of the product's sign, zeros where it is zero
        big = abs(want) > 2.0 ** 129
        assert big.any() and np.array_equal(got[big], np.sign(want[big]) * np.inf)
        assert not got[want == 0].any()
        return
    tol = 4 * U24 * abs(want) + 2.0 ** -133          # bf16's smallest step
    assert (abs(got - want) <= tol + U8 * (abs(want) + tol)).all()
