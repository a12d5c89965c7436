"""Decode of many adapters on a real base whose block scales differ by up to
16 times, at widths whose scales are read each in another way: k a multiple of
1024 (whole slices), of 256 (a ragged last slice), or of 64 only, with and
without double quantisation, on both sides of every change of kernel or layout
(2 to 3 tokens, 8 to 9). The bar is the framework's (2e-2 relative), by token
and by 16 output columns, so that a scale taken from a neighbouring block shows:
among 5 to 33 blocks it moves a value by several times that."""

import numpy as np
import pytest

from _helpers import (bf16_f64, oracle_quant, oracle_wdeq, rel_frob, to_dev, to_host_bits)
from bit_nf4_quantized_19_amd import synth
from oracle import adapters as oad

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from bit_nf4_quantized_19_amd import ops as o
    o.lib()
    return o


@pytest.mark.parametrize("dq", [True, False])
@pytest.mark.parametrize("M", [1, 2, 3, 8, 9, 16])
@pytest.mark.parametrize("d,k,n,r", [(264, 320, 3, 8), (264, 1088, 4, 20), (136, 2112, 3, 16),
                                     (264, 1280, 5, 16), (136, 2048, 4, 33)])
def test_block_scales(ops, d, k, n, r, M, dq):
    print(f"[adapters scales] d={d} k={k} n={n} r={r} M={M} dq={dq}", flush=True)
    rng = np.random.default_rng(M + k)
    W0 = bf16_f64(synth.normal_bf16((d, k), 0.02, 1)).reshape(d, k // 64, 64)
    W0 = W0 * 2.0 ** rng.integers(-2, 3, (d, k // 64, 1))        # exact in bf16
    W0 = (W0.reshape(d, k).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    X = synth.normal_bf16((M, k), 1.0, 2)
    A, B = synth.normal_bf16((n, r, k), k ** -0.5, 3), synth.normal_bf16((n, d, r), 0.02, 4)
    s = rng.uniform(0.25, 1.0, n).astype(np.float32)
    ids = rng.integers(-1, n, M)
    Wd = oracle_wdeq(oracle_quant(W0, dq), d, k)
    want, _ = oad.forward(Wd, *(bf16_f64(v) for v in (X, A, B)), s.astype(np.float64), ids)
    w = ops.quantize(to_dev(W0), dq)
    plan = ops.adapter_plan(torch.from_numpy(ids.astype(np.int32)).cuda(), n)
    Y, _ = ops.linear_fwd_adapters(w, to_dev(X), to_dev(A), to_dev(B), torch.from_numpy(s).cuda(),
                                   plan)
    torch.cuda.synchronize()
    got = bf16_f64(to_host_bits(Y))
    for m in range(M):
        assert rel_frob(got[m], want[m]) <= 2e-2, m
    for c in range(0, d, 16):
        assert rel_frob(got[:, c:c + 16], want[:, c:c + 16]) <= 2e-2, c
