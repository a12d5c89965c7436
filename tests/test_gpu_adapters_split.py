"""Many adapters where the GEMM's tiles share their K-steps among workgroups
(all tiles of a short batch, or those past the last full round of the chip):
a token's values are a function of its own row, its own adapter and the
batch's size, bit for bit, wherever the batch's order puts it."""

import numpy as np
import pytest

from _helpers import bf16_f64, oracle_quant, oracle_wdeq, rel_frob, to_host_bits
from oracle import adapters as oad
from test_gpu_adapters import inputs, on_device, run

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from bit_nf4_quantized_19_amd import ops as o
    o.lib()
    return o


SHAPES = [
    # d, k, M, n, r
    (512, 1024, 5, 3, 16),       # forward by the decode kernels, backward of short tiles
    (520, 1088, 16, 4, 24),
    (1024, 768, 300, 5, 16),     # every tile split, in both directions
    (1024, 1024, 700, 6, 24),
    (1024, 1024, 700, 9, 33),
    (1024, 8704, 1000, 7, 16),   # dX: most tiles whole, the last columns' split
    (8704, 1024, 1000, 7, 40),   # Y: the same
    (6912, 768, 1200, 5, 8),     # Y: 255 whole tiles, no multiple of the eight XCDs
]


@pytest.mark.parametrize("d,k,M,n,r", SHAPES)
def test_batch_order_does_not_change_a_token(ops, d, k, M, n, r):
    print(f"[adapters order] d={d} k={k} M={M} n={n} r={r}", flush=True)
    t = inputs(d, k, M, n, r, "mixed", 13, False)
    a = run(ops, on_device(t))
    perm = np.random.default_rng(1).permutation(M)
    b = run(ops, on_device({key: (v[perm].copy() if key in ("X", "dY", "ids") else v)
                            for key, v in t.items()}))
    p = torch.from_numpy(perm).cuda()
    for name in ("Y", "H", "dX"):
        assert torch.equal(a[name][p], b[name]), name


@pytest.mark.parametrize("d,k,M,n,r", SHAPES)
def test_other_tokens_adapters_do_not_change_a_token(ops, d, k, M, n, r):
    # two in three tokens get other adapters (or none), so that the others lie
    # at other places of the plan, in other tiles and among other runs
    print(f"[adapters others] d={d} k={k} M={M} n={n} r={r}", flush=True)
    t = inputs(d, k, M, n, r, "mixed", 29, False)
    a = run(ops, on_device(t))
    keep = np.arange(M) % 3 == 0
    ids = np.where(keep, t["ids"], np.random.default_rng(2).integers(-1, 2, M))
    b = run(ops, on_device({**t, "ids": ids.astype(np.int32)}))
    at = torch.from_numpy(keep).cuda()
    for name in ("Y", "H", "dX"):
        assert torch.equal(a[name][at], b[name][at]), name


@pytest.mark.parametrize("d,k,M,n,r", [(6912, 768, 1200, 5, 8)])
def test_whole_and_split_columns_against_the_oracle(ops, d, k, M, n, r):
    # the framework's bar, by token and by the 128 columns of a tile
    print(f"[adapters columns] d={d} k={k} M={M} n={n} r={r}", flush=True)
    t = inputs(d, k, M, n, r, "mixed", 37, False)
    got = run(ops, on_device(t))
    Wd = oracle_wdeq(oracle_quant(t["W0"], True), d, k)
    X, A, B, dY = (bf16_f64(t[x]) for x in ("X", "A", "B", "dY"))
    s = t["scale"].astype(np.float64)
    Y, _ = oad.forward(Wd, X, A, B, s, t["ids"])
    dX = oad.backward(Wd, X, A, B, s, t["ids"], dY)[0]
    for name, want in (("Y", Y), ("dX", dX)):
        g = bf16_f64(to_host_bits(got[name]))
        row = np.sqrt(((g - want) ** 2).sum(1) / (want ** 2).sum(1))
        assert row.max() <= 2e-2, name
        for c in range(0, want.shape[1], 128):
            assert rel_frob(g[:, c:c + 128], want[:, c:c + 128]) <= 2e-2, (name, c)
