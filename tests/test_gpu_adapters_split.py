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


SPLIT = [(1024, 768, 300, 5, 16), (1024, 1024, 700, 6, 40), (6912, 768, 1200, 5, 8)]


@pytest.mark.parametrize("d,k,M,n,r", SPLIT)
def test_infinities_stay_with_their_token_and_adapter(ops, d, k, M, n, r):
    print(f"[adapters alone] d={d} k={k} M={M} n={n} r={r}", flush=True)
    t = inputs(d, k, M, n, r, "mixed", 41, False)
    clean = run(ops, on_device(t))
    bad = {key: v.copy() for key, v in t.items()}
    nan, inf = 0x7FC0, 0x7F80
    bad["A"][1, :, ::7], bad["B"][1, ::5, :] = nan, inf
    hit = t["ids"] == 1
    bad["X"][hit], bad["dY"][hit] = inf, nan
    got = run(ops, on_device(bad))
    keep = torch.from_numpy(~hit).cuda()
    for name in ("Y", "H", "dX"):
        assert torch.equal(clean[name][keep], got[name][keep]), name
        assert not torch.isfinite(got[name][~keep].float()).all()
    others = torch.tensor([a for a in range(n) if a != 1], device="cuda")
    for name in ("dA", "dB"):
        assert torch.equal(clean[name][others], got[name][others]), name


@pytest.mark.parametrize("d,k,M,n,r", SPLIT)
def test_two_streams_on_one_plan(ops, d, k, M, n, r):
    # two linears of one batch at once: partial sums, counters and join of each
    # in its own workspace
    print(f"[adapters streams] d={d} k={k} M={M} n={n} r={r}", flush=True)
    lin, plan = [], None
    for i in range(2):
        g = on_device(inputs(d, k, M, n, r, "mixed", 43 + i, False))
        plan = plan or ops.adapter_plan(g["ids"], n)
        w = ops.quantize(g["W0"], True)
        a = dict(w=w, X=g["X"], A=g["A"], B=g["B"], scale=g["scale"], plan=plan)
        Y, H = ops.linear_fwd_adapters(**a)
        want = (Y, H) + ops.linear_bwd_adapters(**a, dY=g["dY"], H=H)
        lin.append((a, g["dY"], want, ops.adapters_workspace(plan, d, k, r, backward=True),
                    torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = []
    for _ in range(6):
        for a, dY, _, ws, st in lin:
            Y, H = ops.linear_fwd_adapters(**a, ws=ws, stream=st)
            got.append((Y, H) + ops.linear_bwd_adapters(**a, dY=dY, H=H, ws=ws, stream=st))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(x, y) for x, y in zip(g, lin[i % 2][2])), i


@pytest.mark.parametrize("d,k,M,n,r", SPLIT)
def test_graph_replay(ops, d, k, M, n, r):
    # plan, forward and backward captured, replayed over a workspace and outputs
    # that hold something else, with the program's own work between
    print(f"[adapters graph] d={d} k={k} M={M} n={n} r={r}", flush=True)
    t = on_device(inputs(d, k, M, n, r, "mixed", 47, False))
    want = run(ops, t)
    w, plan = ops.quantize(t["W0"], True), ops.adapter_plan(t["ids"], n)
    b = {name: torch.empty_like(v) for name, v in want.items()}
    ws = ops.adapters_workspace(plan, d, k, r, backward=True)
    args = (w, t["X"], t["A"], t["B"], t["scale"], plan)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.adapter_plan(t["ids"], n, out=plan)
        ops.linear_fwd_adapters(*args, Y=b["Y"], H=b["H"], ws=ws)
        ops.linear_bwd_adapters(*args, t["dY"], H=b["H"], dX=b["dX"], dA=b["dA"], dB=b["dB"], ws=ws)
    for i in range(4):
        for x in b.values():
            x.fill_(7.0)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(b[x], want[x]) for x in b), i
        assert torch.equal(run(ops, t)["dX"], want["dX"])
