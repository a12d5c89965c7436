"""Many adapters on one base weight against the float64 oracle.

Two comparisons per shape. With an all-zero base only the adapters' terms are
left, and the bound is derived per element: products of bf16 values are exact
in float32, so a sum of c of them in any order is off by at most c 2^-24 of
the sum of magnitudes; s H (s G) enters the matrix units as bf16 high and low
parts, off by 2^-16 of itself; outputs are rounded once (2^-8). With a real
base the bar is the framework's (2e-2 relative Frobenius), row by row, which
also catches a token that got another token's adapter."""

import numpy as np
import pytest

from _helpers import bf16_f64, oracle_quant, oracle_wdeq, rel_frob, to_dev, to_host_bits
from bit_nf4_quantized_19_amd import synth
from oracle import adapters as oad

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

U8, U16, U24 = 2.0 ** -8, 2.0 ** -16, 2.0 ** -24


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from bit_nf4_quantized_19_amd import ops as o
    o.lib()
    return o


def ids_of(pattern, M, n, rng):
    if pattern == "segments":     # runs of one adapter, popularity uneven
        return np.sort(rng.integers(0, n, M))[::-1].copy()
    if pattern == "mixed":
        return rng.integers(-1, n, M)
    if pattern == "none":
        return np.full(M, -1)
    if pattern == "one":
        return np.full(M, n - 1)
    assert pattern == "outside"   # anything outside [0, n) means none
    return rng.choice([0, n - 1, n, n + 1, -1, -(1 << 31), (1 << 31) - 1], M)


def inputs(d, k, M, n, r, pattern, seed, zero_base):
    rng = np.random.default_rng(seed)
    t = {"W0": np.zeros((d, k), np.uint16) if zero_base else synth.normal_bf16((d, k), 0.02, seed),
         "X": synth.normal_bf16((M, k), 1.0, seed + 1),
         "A": synth.normal_bf16((n, r, k), k ** -0.5, seed + 2),
         "B": synth.normal_bf16((n, d, r), 0.1, seed + 3),
         "dY": synth.normal_bf16((M, d), 1.0, seed + 4),
         "scale": rng.uniform(0.25, 4.0, n).astype(np.float32),
         "ids": ids_of(pattern, M, n, rng).astype(np.int32)}
    return t


def on_device(t):
    return {key: (to_dev(v) if v.dtype == np.uint16 else torch.from_numpy(v).cuda())
            for key, v in t.items()}


def run(ops, g, dq=True, n=None):
    w = ops.quantize(g["W0"], dq)
    plan = ops.adapter_plan(g["ids"], g["A"].shape[0])
    Y, H = ops.linear_fwd_adapters(w, g["X"], g["A"], g["B"], g["scale"], plan)
    dX, dA, dB = ops.linear_bwd_adapters(w, g["X"], g["A"], g["B"], g["scale"], plan, g["dY"], H=H)
    torch.cuda.synchronize()
    return {"Y": Y, "H": H, "dX": dX, "dA": dA, "dB": dB}


SHAPES = [
    # d, k, M, n, r, pattern
    (64, 64, 1, 1, 1, "one"),            # the smallest of everything
    (4096, 4096, 1, 8, 16, "mixed"),     # one token (VALU decode)
    (72, 192, 2, 3, 5, "mixed"),         # two tokens, odd rank, ragged k
    (264, 2112, 2, 2, 40, "segments"),   # VALU decode, two slices, r % 16 == 8
    (512, 1088, 7, 5, 16, "mixed"),      # MFMA decode, ragged last slice
    (256, 4160, 3, 2, 128, "outside"),   # largest rank
    (1032, 1024, 16, 1024, 8, "mixed"),  # largest decode batch, most adapters
    (256, 256, 16, 4, 24, "none"),
    (256, 256, 17, 4, 8, "mixed"),       # smallest batch of the GEMM path
    (264, 320, 40, 3, 12, "outside"),
    (1024, 768, 300, 7, 33, "mixed"),    # odd rank, ragged tiles
    (512, 1024, 513, 1000, 4, "mixed"),  # most adapters with no token
    (520, 576, 777, 5, 64, "segments"),
    (256, 512, 1500, 2, 16, "one"),      # an adapter split over token ranges
    (256, 512, 1024, 3, 128, "segments"),
    (128, 256, 90, 4, 16, "none"),
]


@pytest.mark.parametrize("d,k,M,n,r,pattern", SHAPES)
def test_adapter_terms_alone(ops, d, k, M, n, r, pattern):
    print(f"[adapters] d={d} k={k} M={M} n={n} r={r} {pattern}", flush=True)
    t = inputs(d, k, M, n, r, pattern, 100 + M, True)
    got = run(ops, on_device(t))
    X, A, B, dY = (bf16_f64(t[x]) for x in ("X", "A", "B", "dY"))
    s, ids = t["scale"].astype(np.float64), t["ids"]
    W = np.zeros((d, k))
    Y, H = oad.forward(W, X, A, B, s, ids)
    dX, dA, dB = oad.backward(W, X, A, B, s, ids, dY)
    Ha = oad.forward(W, abs(X), abs(A), abs(B), s, ids)[1]    # sums of magnitudes
    eH = 2 * k * U24 * Ha
    assert (abs(got["H"].cpu().numpy() - H) <= eH).all()
    tY, tX = np.zeros((M, d)), np.zeros((M, k))
    tA, tB = np.zeros(A.shape), np.zeros(B.shape)
    for a, rows in enumerate(oad.tokens_of(ids, n)[0]):
        if not rows.size:
            continue
        x, y, ab, bb, c = abs(X[rows]), abs(dY[rows]), abs(A[a]), abs(B[a]), s[a]
        h, eh = abs(H[rows]), eH[rows]
        G, Ga = abs(dY[rows] @ B[a]), y @ bb
        eg = 2 * d * U24 * Ga
        tok = 2 * rows.size + 16          # additions of a token sum, high and low parts
        tY[rows] = c * ((eh + (U16 + 2 * (r + 2) * U24) * h) @ bb.T)
        tX[rows] = c * ((eg + (U16 + 2 * (r + 2) * U24) * G) @ ab)
        tA[a] = c * ((eg + (U16 + tok * U24) * G).T @ x)
        tB[a] = c * (y.T @ (eh + (U16 + tok * U24) * h))
    for name, want, tol in (("Y", Y, tY), ("dX", dX, tX), ("dA", dA, tA), ("dB", dB, tB)):
        g = bf16_f64(to_host_bits(got[name]))
        off = abs(g - want) - (tol + U8 * (abs(want) + tol))
        assert (off <= 0).all(), (name, off.max(), np.argwhere(off > 0)[:4].tolist())


@pytest.mark.parametrize("dq", [True, False])
@pytest.mark.parametrize("d,k,M,n,r,pattern", [
    (4096, 4096, 1, 8, 16, "mixed"), (512, 1088, 7, 5, 16, "mixed"),
    (2048, 4096, 16, 12, 16, "mixed"), (1024, 768, 300, 7, 33, "mixed"),
    (1024, 1024, 700, 3, 16, "segments")])
def test_with_a_real_base(ops, d, k, M, n, r, pattern, dq):
    print(f"[adapters base] d={d} k={k} M={M} n={n} r={r} {pattern} dq={dq}", flush=True)
    t = inputs(d, k, M, n, r, pattern, 300 + M, False)
    got = run(ops, on_device(t), dq)
    Wd = oracle_wdeq(oracle_quant(t["W0"], dq), d, k)
    X, A, B, dY = (bf16_f64(t[x]) for x in ("X", "A", "B", "dY"))
    s = t["scale"].astype(np.float64)
    Y, _ = oad.forward(Wd, X, A, B, s, t["ids"])
    dX, dA, dB = oad.backward(Wd, X, A, B, s, t["ids"], dY)
    for name, want in (("Y", Y), ("dX", dX), ("dA", dA), ("dB", dB)):
        assert rel_frob(bf16_f64(to_host_bits(got[name])), want) <= 2e-2, name
    gY = bf16_f64(to_host_bits(got["Y"]))
    for m in range(M):
        assert rel_frob(gY[m], Y[m]) <= 2e-2, m


def test_one_adapter_is_the_plain_linear(ops):
    # every token on one adapter, in batch order, and enough tiles that none is
    # split over K: the same tiles, sums and roundings as the single-adapter
    # calls, bit for bit
    d, k, M, r, alpha = 4096, 4096, 2040, 16, 32.0
    t = inputs(d, k, M, 1, r, "one", 7, False)
    t["scale"][:] = alpha / r
    g = on_device(t)
    got = run(ops, g)
    w = ops.quantize(g["W0"], True)
    A, B = g["A"][0].contiguous(), g["B"][0].contiguous()
    Y, H = ops.linear_fwd(w, g["X"], A, B, alpha)
    dX, _, _ = ops.linear_bwd(w, g["X"], A, B, alpha, g["dY"], H=H)
    torch.cuda.synchronize()
    assert torch.equal(Y, got["Y"]) and torch.equal(H, got["H"]) and torch.equal(dX, got["dX"])


@pytest.mark.parametrize("M", [3, 16, 200])
def test_tokens_do_not_depend_on_the_others(ops, M):
    # infinities and NaN in one adapter's matrices and tokens leave every
    # other token's values and every other adapter's gradients as they were
    d, k, n, r = 256, 512, 4, 16
    t = inputs(d, k, M, n, r, "mixed", 11, False)
    t["ids"][:3] = (0, 1, -1)
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
    for name in ("dA", "dB"):
        for a in (0, 2, 3):
            assert torch.equal(clean[name][a], got[name][a]), (name, a)


def test_batch_order_does_not_change_a_token(ops):
    d, k, M, n, r = 512, 512, 333, 6, 24
    t = inputs(d, k, M, n, r, "mixed", 13, False)
    a = run(ops, on_device(t))
    perm = np.random.default_rng(1).permutation(M)
    b = run(ops, on_device({key: (v[perm].copy() if key in ("X", "dY", "ids") else v)
                            for key, v in t.items()}))
    p = torch.from_numpy(perm).cuda()
    for name in ("Y", "H", "dX"):
        assert torch.equal(a[name][p], b[name]), name


@pytest.mark.parametrize("M", [1, 9, 130])
def test_recomputed_h_repeats_and_stray_rows(ops, M):
    # H recomputed by the backward gives the saved one's gradients; repeated
    # calls give the same bits; no row past the batch is written; need_dx.
    # Up to 16 tokens the forward sums H in another order than the backward
    # does: both are within 2 k 2^-24 sum |x| |a| of H, so dB differs by at most
    # twice that carried through s |dY|, and by one rounding on each side.
    d, k, n, r = 264, 320, 3, 20
    host = inputs(d, k, M, n, r, "mixed", 17 + M, False)
    t = on_device(host)
    w = ops.quantize(t["W0"], True)
    plan = ops.adapter_plan(t["ids"], n)
    args = (w, t["X"], t["A"], t["B"], t["scale"], plan)
    big = torch.full((M + 4, d), 3.0, dtype=torch.bfloat16, device="cuda")
    bigx = torch.full((M + 4, k), 3.0, dtype=torch.bfloat16, device="cuda")
    Y, H = ops.linear_fwd_adapters(*args, Y=big[:M])
    one = ops.linear_bwd_adapters(*args, t["dY"], H=H, dX=bigx[:M])
    two = ops.linear_bwd_adapters(*args, t["dY"])
    no_dx = ops.linear_bwd_adapters(*args, t["dY"], H=H, need_dx=False)
    Y2, none = ops.linear_fwd_adapters(*args, save_h=False)
    torch.cuda.synchronize()
    assert none is None and no_dx[0] is None and torch.equal(Y, Y2)
    assert bool((big[M:] == 3.0).all()) and bool((bigx[M:] == 3.0).all())
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
    if M > 16:
        assert torch.equal(one[2], two[2])
    else:
        X, A, B, dY = (abs(bf16_f64(host[x])) for x in ("X", "A", "B", "dY"))
        s = host["scale"].astype(np.float64)
        _, Ha = oad.forward(np.zeros((d, k)), X, A, B, s, host["ids"])
        b1, b2 = (bf16_f64(to_host_bits(g[2])) for g in (one, two))
        for a, rows in enumerate(oad.tokens_of(host["ids"], n)[0]):
            tol = 4 * k * U24 * s[a] * (dY[rows].T @ Ha[rows])
            assert (abs(b1[a] - b2[a]) <= tol + U8 * (abs(b1[a]) + abs(b2[a]))).all()
    assert torch.equal(one[1], no_dx[1]) and torch.equal(one[2], no_dx[2])


@pytest.mark.parametrize("M,n", [(1, 1), (5, 3), (64, 1), (1000, 7), (4099, 1024), (70001, 40)])
def test_plan_orders_tokens_by_adapter(ops, M, n):
    rng = np.random.default_rng(M)
    ids = ids_of("mixed", M, n, rng).astype(np.int32)
    plan = ops.adapter_plan(torch.from_numpy(ids).cuda(), n)
    again = ops.adapter_plan(torch.from_numpy(ids).cuda(), n, out=plan)
    torch.cuda.synchronize()
    p = again.data.cpu().numpy().view(np.int32)
    up = lambda x: -(-x // 64) * 64  # noqa: E731
    tok, perm, sid = p[:M], p[up(M):up(M) + M], p[2 * up(M):2 * up(M) + M]
    key = np.where(ids < 0, n, ids)
    assert (tok == ids).all()
    assert (perm == np.argsort(key, kind="stable")).all() and (sid == ids[perm]).all()
    off = p[3 * up(M):3 * up(M) + n + 2]
    assert (off == np.concatenate([[0], np.cumsum(np.bincount(key, minlength=n + 1))])).all()


def test_graph_replay_and_other_stream(ops):
    # plan, forward and backward captured together replay to the eager bits,
    # with the program's own work between; a second stream gives them too
    for M in (5, 150):
        d, k, n, r = 256, 512, 3, 16
        t = on_device(inputs(d, k, M, n, r, "mixed", 23 + M, False))
        want = run(ops, t)
        w = ops.quantize(t["W0"], True)
        plan = ops.adapter_plan(t["ids"], n)
        b = {"Y": torch.empty_like(want["Y"]), "H": torch.empty_like(want["H"]),
             "dX": torch.empty_like(want["dX"]), "dA": torch.empty_like(want["dA"]),
             "dB": torch.empty_like(want["dB"])}
        ws = ops.adapters_workspace(plan, d, k, r, backward=True)

        def step(stream=None):
            ops.adapter_plan(t["ids"], n, out=plan, stream=stream)
            ops.linear_fwd_adapters(w, t["X"], t["A"], t["B"], t["scale"], plan, Y=b["Y"],
                                    H=b["H"], ws=ws, stream=stream)
            ops.linear_bwd_adapters(w, t["X"], t["A"], t["B"], t["scale"], plan, t["dY"], H=b["H"],
                                    dX=b["dX"], dA=b["dA"], dB=b["dB"], ws=ws, stream=stream)

        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        step(s)
        s.synchronize()
        assert all(torch.equal(b[x], want[x]) for x in b)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for i in range(4):
            for x in b.values():
                x.fill_(7.0)
            ws.fill_(255)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(b[x], want[x]) for x in b), i
            assert torch.equal(run(ops, t)["Y"], want["Y"])


def test_refusals(ops):
    t = on_device(inputs(64, 128, 4, 2, 8, "mixed", 1, False))
    w = ops.quantize(t["W0"], True)
    plan = ops.adapter_plan(t["ids"], 2)
    a = dict(w=w, X=t["X"], A=t["A"], B=t["B"], scale=t["scale"], plan=plan)
    for change in (dict(X=t["X"][:3]), dict(X=t["X"].float()), dict(B=t["B"][:1]),
                   dict(A=t["A"][:1]), dict(A=t["A"][0]), dict(scale=t["scale"].double()),
                   dict(scale=t["scale"][:1]), dict(X=t["X"].t().contiguous().t())):
        with pytest.raises(ValueError):
            ops.linear_fwd_adapters(**{**a, **change})
        with pytest.raises(ValueError):
            ops.linear_bwd_adapters(**{**a, **change}, dY=t["dY"])
    with pytest.raises(ValueError):
        ops.linear_fwd_adapters(**a, Y=torch.empty(4, 65, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        ops.linear_bwd_adapters(**a, dY=t["dY"], H=torch.empty(4, 7, device="cuda"))
    with pytest.raises(ValueError):
        ops.adapter_plan(t["ids"].long(), 2)
    with pytest.raises(ValueError):
        ops.adapter_plan(t["ids"], 3, out=plan)
    with pytest.raises(ops.QLoRAError):
        ops.adapter_plan(t["ids"], 1025)
    with pytest.raises(ops.QLoRAError) as e:
        ops.linear_fwd_adapters(**a, ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == ops.QLORA_ERR_WORKSPACE
