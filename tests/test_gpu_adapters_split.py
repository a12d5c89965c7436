"""Many adapters where the GEMM's tiles share their K-steps among workgroups:
a token's values are a function of its own row, its own adapter and the
batch's size, bit for bit, wherever the batch's order puts it."""

import numpy as np
import pytest

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
