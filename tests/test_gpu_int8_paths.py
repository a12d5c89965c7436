"""The 8-bit base where its paths meet: decode with many ranks and with rows that
leave the last workgroup part empty, the two-launch form with many ranks, and
rows that hold a NaN beside it. Bounds as in test_gpu_int8."""

import pytest

from _helpers import to_dev
from test_gpu_int8 import bits, gpu_all, inputs, oracle, within

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from bit_nf4_quantized_19_amd import ops as o
    o.lib()
    return o


@pytest.mark.parametrize("d,k,M,r", [
    # decode: ranks of several waves, of an odd number, and all eight waves'
    (264, 320, 3, 33), (520, 704, 16, 128), (24, 64, 1, 128), (136, 4160, 9, 100),
    # decode of two row blocks a workgroup, the last of 8 or 24 rows
    (8200, 192, 16, 16), (8216, 320, 1, 128), (8232, 64, 5, 12),
    # rows past a workgroup's registers: records and products apart
    (136, 8256, 300, 128), (8264, 192, 300, 100), (16456, 128, 2, 128), (136, 16448, 17, 33)])
def test_against_oracle(ops, d, k, M, r):
    print(f"[int8 paths] d={d} k={k} M={M} r={r}", flush=True)
    W, X, dY, A, B = inputs(d, k, M, r, seed=M + r)
    want, tol = oracle(W, X, dY, A, B, 2.0)
    w, Y, H, dX, dA, dB = gpu_all(ops, W, X, dY, A, B, 2.0 * r)
    assert (abs(H.cpu().numpy() - want["H"]) <= tol["H"]).all()
    for name, got in (("Y", Y), ("dX", dX), ("dA", dA), ("dB", dB)):
        within(bits(got), want[name], tol[name], name)
    again = ops.linear_bwd_int8(w, *(to_dev(v) for v in (X, A, B)), 2.0 * r, to_dev(dY))
    for g, v in zip(again, (dX, dA, dB)):
        assert torch.equal(g, v)


@pytest.mark.parametrize("d,k,M", [(136, 8256, 300), (8264, 192, 300), (136, 16448, 17),
                                   (8200, 192, 5), (264, 320, 1100)])
def test_rows_do_not_reach_each_other(ops, d, k, M):
    print(f"[int8 paths, rows] d={d} k={k} M={M}", flush=True)
    W, X, dY, A, B = inputs(d, k, M, 20, seed=3)
    _, Y, H, dX, _, _ = gpu_all(ops, W, X, dY, A, B, 40.0)
    bad = [1, M - 1]
    X2, dY2 = X.copy(), dY.copy()
    X2[1, 3], X2[M - 1, k - 1] = 0x7FC0, 0x7F80
    dY2[1, d - 1], dY2[M - 1, 0] = 0xFF80, 0x7FC0
    _, Y2, H2, dX2, _, _ = gpu_all(ops, W, X2, dY2, A, B, 40.0)
    keep = torch.tensor([i for i in range(M) if i not in bad], device="cuda")
    for got, clean in ((Y2, Y), (H2, H), (dX2, dX)):
        assert torch.equal(got[keep], clean[keep])
    assert torch.isnan(Y2[bad]).all() and torch.isnan(dX2[bad]).all()
