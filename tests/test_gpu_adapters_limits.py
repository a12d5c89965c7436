"""Many adapters and token log probabilities where calls meet or sizes grow:
matrices past 2^32 bytes, tiles past the last full round, two streams at once
on one plan, outputs that lack what was asked. Bounds as in test_gpu_adapters.py: sums of c exact products
off by at most c 2^-24 of their magnitudes, high and low parts by 2^-16,
outputs rounded once (2^-8)."""

import numpy as np
import pytest

from _helpers import (bf16_f64, oracle_quant, oracle_wdeq, rel_frob, to_dev, to_host_bits)
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


def bits(t):
    return bf16_f64(to_host_bits(t))


def within(got, want, tol, name):
    off = abs(got - want) - (tol + U8 * (abs(want) + tol))
    assert (off <= 0).all(), (name, off.max())


def test_offsets_past_32_bits(ops):
    # tokens and adapters whose elements lie past 2^31 of their matrix; all
    # other rows and matrices are zero and must stay so in the results
    d, k, M, n, r = 128, 16896, 140000, 1024, 128
    print(f"[adapters long] d={d} k={k} M={M} n={n} r={r}", flush=True)
    used = [0, 517, 1023]
    rows = np.array([0, 1, 2, 70000, 70001, 127100, 127101, 139990, 139995, 139997, 139998, 139999])
    of = np.array([0, 2, 1, 2, 0, 2, 1, 1, 2, 0, -1, 2])     # index into used
    assert (M - 1) * k > 1 << 31 and used[2] * r * k > 1 << 31
    bf, dev = torch.bfloat16, "cuda"

    def rand(shape, scale, seed):
        g = torch.Generator(device=dev).manual_seed(seed)
        return (torch.randn(shape, generator=g, device=dev) * scale).to(bf)

    x, y = rand((rows.size, k), 1.0, 1), rand((rows.size, d), 1.0, 2)
    A, B = torch.zeros(n, r, k, dtype=bf, device=dev), torch.zeros(n, d, r, dtype=bf, device=dev)
    A[used], B[used] = rand((3, r, k), k ** -0.5, 3), rand((3, d, r), 0.1, 4)
    X, dY = torch.zeros(M, k, dtype=bf, device=dev), torch.zeros(M, d, dtype=bf, device=dev)
    rt = torch.from_numpy(rows).to(dev)
    X[rt], dY[rt] = x, y
    scale = torch.linspace(0.5, 2.0, n, device=dev)
    ids = (torch.arange(M, device=dev) % (n + 1) - 1).int()
    ids[rt] = torch.tensor([used[i] if i >= 0 else -1 for i in of], dtype=torch.int32, device=dev)
    w = ops.quantize(torch.zeros(d, k, dtype=bf, device=dev), True)

    xs, ys, As, Bs = bits(x), bits(y), bits(A[used]), bits(B[used])
    s = scale[used].cpu().numpy().astype(np.float64)
    W = np.zeros((d, k))
    Yw, Hw = oad.forward(W, xs, As, Bs, s, of)
    dXw, dAw, dBw = oad.backward(W, xs, As, Bs, s, of, ys)
    eH = 2 * k * U24 * oad.forward(W, abs(xs), abs(As), abs(Bs), s, of)[1]
    tY, tX, tA, tB = (np.zeros(v.shape) for v in (Yw, dXw, dAw, dBw))
    for a in range(3):
        i = np.flatnonzero(of == a)
        h, G, Ga = abs(Hw[i]), abs(ys[i] @ Bs[a]), abs(ys[i]) @ abs(Bs[a])
        eg, tok = 2 * d * U24 * Ga, 2 * i.size + 16
        tY[i] = s[a] * ((eH[i] + (U16 + 2 * (r + 2) * U24) * h) @ abs(Bs[a]).T)
        tX[i] = s[a] * ((eg + (U16 + 2 * (r + 2) * U24) * G) @ abs(As[a]))
        tA[a] = s[a] * ((eg + (U16 + tok * U24) * G).T @ abs(xs[i]))
        tB[a] = s[a] * (abs(ys[i]).T @ (eH[i] + (U16 + tok * U24) * h))

    plan = ops.adapter_plan(ids, n)
    Y, H = ops.linear_fwd_adapters(w, X, A, B, scale, plan)
    dX, dA, dB = ops.linear_bwd_adapters(w, X, A, B, scale, plan, dY, H=H)
    torch.cuda.synchronize()
    within(bits(Y[rt]), Yw, tY, "Y")
    within(bits(dX[rt]), dXw, tX, "dX")
    within(bits(dA[used]), dAw, tA, "dA")
    within(bits(dB[used]), dBw, tB, "dB")
    for t in (Y, dX):
        t[rt] = 0
        assert not bool(t.any())
    for t in (dA, dB):
        t[used] = 0
        assert not bool(t.any())
    del dX, dA, dB, Y, X
    for m in (2, 7, 12):                    # the decode kernels on the same adapters
        p = ops.adapter_plan(ids[rt[-m:]].contiguous(), n)
        Y, _ = ops.linear_fwd_adapters(w, x[-m:].contiguous(), A, B, scale, p)
        within(bits(Y), Yw[-m:], tY[-m:], ("decode", m))


@pytest.mark.parametrize("d,k,M,n,r", [(2048, 11008, 777, 5, 12), (11008, 2176, 800, 6, 40)])
def test_tiles_past_the_last_full_round(ops, d, k, M, n, r):
    # 344 tiles (of dX; of Y) for 256 compute units: some whole, the rest split
    print(f"[adapters rounds] d={d} k={k} M={M} n={n} r={r}", flush=True)
    rng = np.random.default_rng(M)
    bf = lambda shape, scale, seed: synth.normal_bf16(shape, scale, seed)   # noqa: E731
    W0, X, dY = bf((d, k), 0.02, 1), bf((M, k), 1.0, 2), bf((M, d), 1.0, 3)
    A, B = bf((n, r, k), k ** -0.5, 4), bf((n, d, r), 0.1, 5)
    s, ids = rng.uniform(0.25, 4.0, n).astype(np.float32), rng.integers(-1, n, M)
    Wd = oracle_wdeq(oracle_quant(W0, True), d, k)
    f = [bf16_f64(v) for v in (X, A, B, dY)]
    Yw, _ = oad.forward(Wd, f[0], f[1], f[2], s.astype(np.float64), ids)
    dXw, dAw, dBw = oad.backward(Wd, f[0], f[1], f[2], s.astype(np.float64), ids, f[3])
    gX, gA, gB, gY = (to_dev(v) for v in (X, A, B, dY))
    gs, gi = torch.from_numpy(s).cuda(), torch.from_numpy(ids.astype(np.int32)).cuda()
    w, plan = ops.quantize(to_dev(W0), True), ops.adapter_plan(gi, n)
    first = None
    for _ in range(2):
        Y, H = ops.linear_fwd_adapters(w, gX, gA, gB, gs, plan)
        got = (Y,) + ops.linear_bwd_adapters(w, gX, gA, gB, gs, plan, gY, H=H)
        torch.cuda.synchronize()
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(got, first))
    for name, g, want in zip(("Y", "dX", "dA", "dB"), got, (Yw, dXw, dAw, dBw)):
        assert rel_frob(bits(g), want) <= 2e-2, name
    for g, want in ((bits(got[0]), Yw), (bits(got[1]), dXw)):
        row = np.sqrt(((g - want) ** 2).sum(1) / (want ** 2).sum(1))
        assert row.max() <= 2e-2
        for c in range(0, want.shape[1], 128):   # a tile's columns
            assert rel_frob(g[:, c:c + 128], want[:, c:c + 128]) <= 2e-2, c


@pytest.mark.parametrize("d,k,M,n,r", [
    (1024, 11008, 16, 5, 64),      # H's pieces taken in turn, a last turn not full
    (1024, 11008, 8, 3, 128),
    (2912, 22016, 11, 4, 16),      # row workgroups of more than one round
    (2912, 22016, 5, 4, 40)])
def test_decode_h_workgroups(ops, d, k, M, n, r):
    print(f"[adapters decode] d={d} k={k} M={M} n={n} r={r}", flush=True)
    rng = np.random.default_rng(M)
    W0, X = synth.normal_bf16((d, k), 0.02, 1), synth.normal_bf16((M, k), 1.0, 2)
    A, B = synth.normal_bf16((n, r, k), k ** -0.5, 3), synth.normal_bf16((n, d, r), 0.1, 4)
    s, ids = rng.uniform(0.25, 4.0, n).astype(np.float32), rng.integers(-1, n, M)
    gi = torch.from_numpy(ids.astype(np.int32)).cuda()
    w, plan = ops.quantize(to_dev(W0), True), ops.adapter_plan(gi, n)
    H = torch.full((M, r), float("nan"), device="cuda")
    Y, H = ops.linear_fwd_adapters(w, to_dev(X), to_dev(A), to_dev(B), torch.from_numpy(s).cuda(),
                                   plan, H=H)
    torch.cuda.synchronize()
    Wd = oracle_wdeq(oracle_quant(W0, True), d, k)
    x, a, b = bf16_f64(X), bf16_f64(A), bf16_f64(B)
    Yw, Hw = oad.forward(Wd, x, a, b, s.astype(np.float64), ids)
    Ha = oad.forward(np.zeros((d, k)), abs(x), abs(a), abs(b), s.astype(np.float64), ids)[1]
    assert (abs(H.cpu().numpy() - Hw) <= 2 * k * U24 * Ha).all()
    got = bits(Y)
    for m in range(M):
        assert rel_frob(got[m], Yw[m]) <= 2e-2, m


@pytest.mark.parametrize("M", [9, 14, 300])
def test_two_streams_share_a_plan(ops, M):
    # two linears of one batch at once, each with its own workspace, on one plan
    d, k, n, r = 512, 1024, 5, 16
    dev = "cuda"

    def data(shape, scale, seed):
        return torch.from_numpy(synth.normal_bf16(shape, scale, seed).view(np.int16)).to(dev).view(
            torch.bfloat16)

    ids = (torch.arange(M, device=dev) * 7 % (n + 1) - 1).int()
    scale = torch.ones(n, device=dev)
    plan = ops.adapter_plan(ids, n)
    lin = []
    for i in range(2):
        w = ops.quantize(data((d, k), 0.02, 10 * i + 1), True)
        a = dict(w=w, X=data((M, k), 1.0, 10 * i + 2), A=data((n, r, k), k ** -0.5, 10 * i + 3),
                 B=data((n, d, r), 0.1, 10 * i + 4), scale=scale, plan=plan)
        dY = data((M, d), 1.0, 10 * i + 5)
        Y, H = ops.linear_fwd_adapters(**a)
        want = (Y, H) + ops.linear_bwd_adapters(**a, dY=dY, H=H)
        lin.append((a, dY, want, ops.adapters_workspace(plan, d, k, r, backward=True),
                    torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = []
    for _ in range(8):
        for a, dY, _, ws, st in lin:
            Y, H = ops.linear_fwd_adapters(**a, ws=ws, stream=st)
            got.append((Y, H) + ops.linear_bwd_adapters(**a, dY=dY, H=H, ws=ws, stream=st))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(x, y) for x, y in zip(g, lin[i % 2][2])), i


def test_alternatives_need_their_outputs(ops):
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    t = torch.zeros(4, dtype=torch.int64, device="cuda")
    out = ops.TokenLogprobs.empty(4)
    ops.token_logprobs(x, t, out=out)
    with pytest.raises(ValueError):
        ops.token_logprobs(x, t, top=2, out=out)
    with pytest.raises(ValueError):
        ops.token_logprobs(x, t, top=2, out=ops.TokenLogprobs.empty(4, 3))


def test_other_devices_are_refused(ops):
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    t = torch.zeros(4, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError):
        ops.token_logprobs(x, t, top=2, ws=torch.empty(1 << 16, dtype=torch.uint8))
    with pytest.raises(ValueError):
        ops.token_logprobs(x, t.cpu())
    ids = torch.zeros(4, dtype=torch.int32, device="cuda")
    plan = ops.adapter_plan(ids, 2)
    away = ops.AdapterPlan(4, 2, plan.data.cpu())
    with pytest.raises(ValueError):
        ops.adapter_plan(ids, 2, out=away)
    w = ops.quantize(torch.zeros(64, 64, dtype=torch.bfloat16, device="cuda"), True)
    a = dict(w=w, X=x, A=torch.zeros(2, 8, 64, dtype=torch.bfloat16, device="cuda"),
             B=torch.zeros(2, 64, 8, dtype=torch.bfloat16, device="cuda"),
             scale=torch.ones(2, device="cuda"), plan=plan)
    ws = torch.empty(1 << 20, dtype=torch.uint8)
    for bad in (dict(plan=away), dict(ws=ws)):
        with pytest.raises(ValueError):
            ops.linear_fwd_adapters(**{**a, **bad})
        with pytest.raises(ValueError):
            ops.linear_bwd_adapters(**{**a, **bad}, dY=x)
