"""Low-rank adapters of many requests: plan, forward and gradients against the fp64 oracle.

Tolerances, from the arithmetic: bf16 products are exact in fp32, and a sum of n of them is off by at most
depth * 2^-23 * (the sum of magnitudes), depth = the additions one result goes through: n / 16 mma steps of
one accumulator at most, and 64 for the joins of warps, CTAs and slices.  h and dh enter a product with a bf16 result
as two bf16 terms, which leaves 2^-17 of them, and as three where the result is fp32.  The result is rounded once, half
a step of its type.
"""
import numpy as np
import pytest
import torch

import grouped_gemm_03_b200 as gg
from oracle import as_f64, tuning

pytestmark = pytest.mark.gpu
DEV = "cuda"
STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
SPLIT = 2.0 ** -17


def depth(n):
    return (n / 16 + 64) * 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def _built():
    from grouped_gemm_03_b200.build import build
    build()


def _bf(r, *shape, std=1.0):
    return torch.from_numpy(r.normal(size=shape) * std).to(torch.bfloat16)


def _inputs(rows, n, d, N, R, seed=0, bare=True, only=None):
    r = np.random.default_rng(seed)
    row = r.integers(-1 if bare else 0, n, size=rows).astype(np.int32)
    if only is not None:
        row = r.choice(np.array(only, np.int32), size=rows)
    return dict(row=row, x=_bf(r, rows, d), A=_bf(r, n, R, d, std=d ** -0.5), B=_bf(r, n, N, R, std=0.2),
                scale=torch.from_numpy(r.uniform(0.5, 2, size=n).astype(np.float32)), base=_bf(r, rows, N),
                dC=_bf(r, rows, N), dx_base=_bf(r, rows, d))


def _gpu(s, *names):
    return [s[n].to(DEV) for n in names]


def _plan(s, n):
    return gg.adapter_plan(torch.from_numpy(s["row"]).to(DEV), n)


def _close(got, want, tol, what):
    got = as_f64(got)
    tol = tol + 1e-30
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3], got[bad][:3], want[bad][:3], tol[bad][:3])


def _check_forward(s, out, h, scale, base):
    n = len(s["A"])
    want, wh = tuning.lora(s["x"], s["A"], s["B"], s["row"], scale, base)
    ax, aA, aB = (np.abs(as_f64(s[v])) for v in ("x", "A", "B"))
    mag, magh = tuning.lora(ax, aA, aB, s["row"], None if scale is None else scale.abs(),
                            None if base is None else base.abs())
    R, d = s["A"].shape[1:]
    eh = depth(d) * magh
    if h is not None:
        _close(h, wh, eh, "h")
    tol = np.zeros_like(want)
    for a in range(n):
        r = np.nonzero(s["row"] == a)[0]
        sc = 1.0 if scale is None else abs(float(scale[a]))
        tol[r] = sc * ((eh[r] + (SPLIT + 2.0 ** -23) * np.abs(wh[r])) @ aB[a].T)
        hb = sc * np.abs(wh[r]) @ aB[a].T + (0 if base is None else np.abs(as_f64(base))[r])
        tol[r] += depth(2 * R) * hb
    _close(out, want, tol + STEP[out.dtype] * (np.abs(want) + tol), "out")


SHAPES = [(1, 1, 8, 8, 8), (1, 3, 64, 24, 16), (15, 2, 40, 200, 8), (16, 1, 32, 32, 16), (17, 5, 264, 72, 24),
          (61, 48, 512, 704, 16), (64, 2, 256, 256, 32), (65, 1, 1032, 136, 64), (130, 7, 128, 1000, 40),
          (200, 3, 1408, 2048, 8), (333, 4, 96, 96, 128), (515, 2, 512, 264, 16), (700, 40, 200, 328, 64),
          (1100, 3, 64, 128, 104), (40, 1024, 64, 64, 8), (2100, 100, 32, 40, 16), (1300, 1, 2056, 512, 32)]


@pytest.mark.parametrize("rows", [0, 1, 31, 1000, 1024, 1025, 5000, 140000])
@pytest.mark.parametrize("n", [1, 7, 1023, 1024])
def test_plan(rows, n):
    row = np.random.default_rng(rows + n).integers(-1, n, size=rows).astype(np.int32)
    offsets, order = gg.adapter_plan(torch.from_numpy(row).to(DEV), n)
    key = np.where(row < 0, n, row)
    assert np.array_equal(order.cpu().numpy(), np.argsort(key, kind="stable"))
    assert np.array_equal(offsets.cpu().numpy(), np.searchsorted(np.sort(key), np.arange(n + 1)))


def test_plan_reports_wrong_ids():
    ws = torch.empty(gg.lib().moe_adapter_plan_workspace_size(6, 3), dtype=torch.uint8, device=DEV)
    row = torch.tensor([0, 3, 2, -2, -1, 0], dtype=torch.int32, device=DEV)
    offsets, order = gg.adapter_plan(row, 3, ws=ws)
    assert gg.read_device_status(ws) == -1
    assert offsets.tolist() == [0, 2, 2, 3] and order.tolist() == [0, 5, 2, 1, 3, 4]
    gg.adapter_plan(row.clamp(-1, 2), 3, ws=ws)
    assert gg.read_device_status(ws) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,n,d,N,R", SHAPES)
def test_forward(rows, n, d, N, R, dtype):
    s = _inputs(rows, n, d, N, R, seed=rows)
    x, A, B, scale = _gpu(s, "x", "A", "B", "scale")
    base = s["base"].to(dtype)
    off, order = _plan(s, n)
    out, h = gg.lora(x, A, B, off, order, scale=scale, base=base.to(DEV), want_h=True)
    assert out.dtype == dtype
    _check_forward(s, out, h, s["scale"], base)
    # in place, and without h: the same bits; rows without an adapter are left as they were
    y = base.to(DEV)
    assert gg.lora(x, A, B, off, order, scale=scale, base=y, out=y) is y
    assert torch.equal(y, out)
    # no base, no scale
    _check_forward(s, gg.lora(x, A, B, off, order, out_dtype=dtype), None, None, None)


def _check_backward(s, got, h, scale, dx_base):
    n, R, d = s["A"].shape
    rows, N = s["dC"].shape
    dx, dA, dB = got
    wx, wA, wB = tuning.lora_backward(s["dC"], s["x"], h, s["A"], s["B"], s["row"], scale, dx_base)
    ac, ax, ah, aA, aB = (np.abs(as_f64(v)) for v in (s["dC"], s["x"], h, s["A"], s["B"]))
    tx = np.zeros_like(wx)
    for a in range(n):
        r = np.nonzero(s["row"] == a)[0]
        sc = 1.0 if scale is None else abs(float(scale[a]))
        mdh = sc * ac[r] @ aB[a]
        edh = (depth(N) + SPLIT + 2.0 ** -22) * mdh
        tx[r] = edh @ aA[a] + depth(2 * R) * (mdh @ aA[a])
        if dx_base is not None:
            tx[r] += depth(0) * np.abs(as_f64(dx_base))[r]
        if dA is not None:
            ta = edh.T @ ax[r] + depth(2 * len(r)) * (mdh.T @ ax[r])
            _close(dA[a], wA[a], ta + STEP[dA.dtype] * (np.abs(wA[a]) + ta), f"dA {a}")
            tb = (depth(2 * len(r)) + SPLIT + 2.0 ** -22) * sc * (ac[r].T @ ah[r])
            _close(dB[a], wB[a], tb + STEP[dB.dtype] * (np.abs(wB[a]) + tb), f"dB {a}")
    if dx is not None:
        _close(dx, wx, tx + STEP[dx.dtype] * (np.abs(wx) + tx), "dx")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,n,d,N,R", SHAPES)
def test_backward(rows, n, d, N, R, dtype):
    s = _inputs(rows, n, d, N, R, seed=rows + 1)
    h = torch.from_numpy(np.random.default_rng(5).normal(size=(rows, R)).astype(np.float32))
    dC, x, A, B, scale = _gpu(s, "dC", "x", "A", "B", "scale")
    base = s["dx_base"].to(dtype)
    off, order = _plan(s, n)
    got = gg.lora_backward(dC, x, h.to(DEV), A, B, off, order, scale=scale, dx_base=base.to(DEV), grad_dtype=dtype)
    assert got[0].dtype == dtype and got[1].dtype == dtype
    _check_backward(s, got, h, s["scale"], base)
    again = gg.lora_backward(dC, x, h.to(DEV), A, B, off, order, scale=scale, dx_base=base.to(DEV), grad_dtype=dtype)
    assert all(torch.equal(u, v) for u, v in zip(got, again))
    # in place
    y = base.to(DEV)
    assert torch.equal(gg.lora_backward(dC, x, h.to(DEV), A, B, off, order, scale=scale, dx_base=y, dx=y,
                                        want_grads=False)[0], got[0])
    # no base, no scale, dx alone and gradients alone
    dx = gg.lora_backward(dC, x, h.to(DEV), A, B, off, order, want_grads=False, dx_dtype=dtype)[0]
    dA, dB = gg.lora_backward(dC, x, h.to(DEV), A, B, off, order, want_dx=False)[1:]
    _check_backward(s, (dx, dA, dB), h, None, None)


def test_many_rows_of_one_adapter_and_none_of_others():
    s = _inputs(3000, 6, 136, 72, 16, seed=3, only=[4, 4, 4, 1, -1])
    x, A, B, scale, dC = _gpu(s, "x", "A", "B", "scale", "dC")
    off, order = _plan(s, 6)
    out, h = gg.lora(x, A, B, off, order, scale=scale, want_h=True)
    _check_forward(s, out, h, s["scale"], None)
    got = gg.lora_backward(dC, x, h, A, B, off, order, scale=scale)
    _check_backward(s, got, h.cpu(), s["scale"], None)
    for a in (0, 2, 3, 5):
        assert not got[1][a].any() and not got[2][a].any()
    assert not h[torch.from_numpy(s["row"]).to(DEV) < 0].any()


def test_no_rows_and_no_adapted_rows():
    s = _inputs(20, 3, 64, 48, 8, seed=4, only=[-1])
    x, A, B, base, dC = _gpu(s, "x", "A", "B", "base", "dC")
    off, order = _plan(s, 3)
    assert torch.equal(gg.lora(x, A, B, off, order, base=base), base)
    assert not gg.lora(x, A, B, off, order).any()
    dx, dA, dB = gg.lora_backward(dC, x, torch.zeros(20, 8, device=DEV), A, B, off, order, dx_base=x.clone())
    assert torch.equal(dx, x) and not dA.any() and not dB.any()
    off, order = gg.adapter_plan(torch.empty(0, dtype=torch.int32, device=DEV), 3)
    assert gg.lora(x[:0], A, B, off, order).shape == (0, 48)
    dx, dA, dB = gg.lora_backward(dC[:0], x[:0], torch.zeros(0, 8, device=DEV), A, B, off, order)
    assert dx.shape == (0, 64) and not dA.any() and not dB.any()


def test_not_finite_rows_stay_their_own():
    s = _inputs(90, 2, 64, 64, 16, seed=5)
    s["x"][13] = float("inf")
    s["x"][14, 3] = float("nan")
    s["row"][13], s["row"][14] = 0, -1
    x, A, B, base = _gpu(s, "x", "A", "B", "base")
    off, order = _plan(s, 2)
    out = gg.lora(x, A, B, off, order, base=base)
    assert not torch.isfinite(out[13]).any() and torch.equal(out[14], base[14])
    keep = [i for i in range(90) if i not in (13, 14)]
    assert torch.isfinite(out[keep]).all()


def test_entries_that_name_no_row_are_skipped():
    # in bounds by the kernel's own checks: an id outside the rows reads nothing and writes nothing
    s = _inputs(40, 2, 64, 64, 8, seed=6, bare=False)
    x, A, B, base, dC = _gpu(s, "x", "A", "B", "base", "dC")
    off, order = _plan(s, 2)
    lost = order[[3, 30]].tolist()
    bad = order.clone()
    bad[3], bad[30] = -1, 40
    good = gg.lora(x, A, B, off, order, base=base)
    out = base.clone()
    gg.lora(x, A, B, off, bad, base=out, out=out)
    keep = [i for i in range(40) if i not in lost]
    assert torch.equal(out[keep], good[keep]) and torch.equal(out[lost], base[lost])
    h = torch.randn(40, 8, device=DEV)
    dx = x.float()
    full = gg.lora_backward(dC, x, h, A, B, off, order, dx_base=x.float())[0]
    gg.lora_backward(dC, x, h, A, B, off, bad, dx_base=dx, dx=dx)
    assert torch.equal(dx[keep], full[keep]) and torch.equal(dx[lost], x.float()[lost])


def test_captured_and_replayed_with_another_batch():
    n, d, N, R, rows = 4, 128, 192, 16, 150
    s = _inputs(rows, n, d, N, R, seed=7)
    x, A, B, scale, base, dC = _gpu(s, "x", "A", "B", "scale", "base", "dC")
    row = torch.from_numpy(s["row"]).to(DEV)
    ws = torch.empty(gg.lib().moe_lora_backward_workspace_size(rows, n, d, N, R), dtype=torch.uint8, device=DEV)

    def step():
        off, order = gg.adapter_plan(row, n)
        out, h = gg.lora(x, A, B, off, order, scale=scale, base=base, want_h=True)
        return (out, h) + gg.lora_backward(dC, x, h, A, B, off, order, scale=scale, ws=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    graphs = []
    for _ in range(2):   # two graphs that share the workspace, replayed one after the other
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            graphs.append((graph, step()))
    for seed in (8, 9):
        t = _inputs(rows, n, d, N, R, seed=seed)
        row.copy_(torch.from_numpy(t["row"]))
        x.copy_(t["x"])
        for graph, got in graphs:
            graph.replay()
            torch.cuda.synchronize()
            for u, v in zip(got, step()):
                assert torch.equal(u, v)
        t.update(A=s["A"], B=s["B"], dC=s["dC"])
        _check_forward(t, got[0], got[1], s["scale"], s["base"])
        _check_backward(t, got[2:], got[1].cpu(), s["scale"], None)


def test_two_calls_at_once_on_two_streams():
    jobs = []
    for seed in (1, 2):
        s = _inputs(900, 3, 512, 640, 32, seed=seed)
        jobs.append((s, _plan(s, 3), _gpu(s, "x", "A", "B", "dC"), torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = []
    for s, (off, order), (x, A, B, dC), stream in jobs:
        out, h = gg.lora(x, A, B, off, order, want_h=True, stream=stream)
        got.append((out, h, gg.lora_backward(dC, x, h, A, B, off, order, stream=stream)))
    torch.cuda.synchronize()
    for (s, *_), (out, h, grads) in zip(jobs, got):
        _check_forward(s, out, h, None, None)
        _check_backward(s, grads, h.cpu(), None, None)


def test_rows_past_32_bit_offsets():
    # 2^31 elements of out before the last rows: addresses need 64 bits, in one launch and in two
    for rows, N, d, R in ((300000, 7168, 8, 8), (40000, 504, 57344, 16)):
        _rows_past_32_bit_offsets(rows, N, d, R)


def _rows_past_32_bit_offsets(rows, N, d, R):
    x = torch.zeros(rows, d, dtype=torch.bfloat16, device=DEV)
    x[-3:] = 1
    A = torch.ones(1, R, d, dtype=torch.bfloat16, device=DEV)
    B = torch.ones(1, N, R, dtype=torch.bfloat16, device=DEV)
    row = torch.full((rows,), -1, dtype=torch.int32, device=DEV)
    row[-3:] = 0
    off, order = gg.adapter_plan(row, 1)
    out = torch.zeros(rows, N, dtype=torch.bfloat16, device=DEV)
    gg.lora(x, A, B, off, order, base=out, out=out)
    assert (out[-3:] == d * R).all() and not out[:-3].any()


# sizes at which the forward's products are launches of their own: ragged and empty adapters, odd widths
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,n,d,N,R,only", [(40000, 1, 1032, 1000, 16, None), (26000, 4, 520, 504, 24, [0, 0, 0, 3, -1]),
                                               (12500, 5, 520, 504, 64, None), (6100, 2, 264, 248, 128, [-1, 1, 1, 1]),
                                               (6100, 3, 256, 264, 104, None)])
def test_two_launches(rows, n, d, N, R, only, dtype):
    assert gg.lib().moe_lora_workspace_size(rows, n, d, N, R) > 0
    s = _inputs(rows, n, d, N, R, seed=R, only=only)
    x, A, B, scale = _gpu(s, "x", "A", "B", "scale")
    base = s["base"].to(dtype)
    off, order = _plan(s, n)
    out, h = gg.lora(x, A, B, off, order, scale=scale, base=base.to(DEV), want_h=True)
    _check_forward(s, out, h, s["scale"], base)
    y = base.to(DEV)
    assert torch.equal(gg.lora(x, A, B, off, order, scale=scale, base=y, out=y), out)   # in place, without h
    bare = torch.from_numpy(s["row"]).to(DEV) < 0
    assert not h[bare].any()
    plain = gg.lora(x, A, B, off, order, out_dtype=dtype)
    _check_forward(s, plain, None, None, None)
    # entries that name no row are skipped, values that are not finite stay their own
    bad = order.clone()
    bad[3] = rows + 5
    z = base.to(DEV)
    gg.lora(x, A, B, off, bad, scale=scale, base=z, out=z)
    keep = torch.ones(rows, dtype=torch.bool, device=DEV)
    keep[order[3].long()] = False
    assert torch.equal(z[keep], out[keep]) and torch.equal(z[~keep], base.to(DEV)[~keep])
    mine = torch.from_numpy(s["row"]).to(DEV) == n - 1
    x[mine], A[n - 1], B[n - 1] = float("nan"), float("inf"), float("nan")
    odd = gg.lora(x, A, B, off, order, out_dtype=dtype)
    assert torch.equal(odd[~mine], plain[~mine]) and not torch.isfinite(odd[mine]).any()


# gradients of few rows to an adapter, in one launch: alone, ragged (some of more tiles than one), every rank
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,n,d,N,R,only", [(1, 1, 8, 8, 8, None), (4, 1, 4096, 136, 32, None), (3, 2, 72, 1032, 24, [1]),
                                               (61, 48, 264, 520, 16, None), (100, 100, 520, 264, 64, None),
                                               (160, 40, 136, 2056, 104, [0, 0, 0, 5, 39, -1]), (32, 8, 648, 72, 40, [7]),
                                               (200, 1024, 64, 64, 8, None), (33, 9, 2048, 2816, 128, None)])
def test_backward_of_few_rows(rows, n, d, N, R, only, dtype):
    s = _inputs(rows, n, d, N, R, seed=rows + R, only=only)
    h = torch.from_numpy(np.random.default_rng(6).normal(size=(rows, R)).astype(np.float32))
    dC, x, A, B, scale = _gpu(s, "dC", "x", "A", "B", "scale")
    base = s["dx_base"].to(dtype)
    off, order = _plan(s, n)
    ws = torch.empty(gg.lib().moe_lora_backward_workspace_size(rows, n, d, N, R), dtype=torch.uint8, device=DEV)
    ws.fill_(0xff)
    got = gg.lora_backward(dC, x, h.to(DEV), A, B, off, order, scale=scale, dx_base=base.to(DEV), grad_dtype=dtype, ws=ws)
    assert gg.read_device_status(ws) == 0
    _check_backward(s, got, h, s["scale"], base)
    y = base.to(DEV)
    assert torch.equal(gg.lora_backward(dC, x, h.to(DEV), A, B, off, order, scale=scale, dx_base=y, dx=y,
                                        want_grads=False)[0], got[0])
    dx = gg.lora_backward(dC, x, h.to(DEV), A, B, off, order, want_grads=False, dx_dtype=dtype)[0]
    dA, dB = gg.lora_backward(dC, x, h.to(DEV), A, B, off, order, want_dx=False)[1:]
    _check_backward(s, (dx, dA, dB), h, None, None)


# adapters of several chunks of a gradient
@pytest.mark.parametrize("rows,n,d,N,R,only", [(2600, 2, 512, 392, 16, [0]), (2600, 3, 264, 512, 32, [0, 0, 2]),
                                               (3100, 2, 1160, 648, 64, [1]), (2300, 2, 256, 384, 128, [0, 0, 1])])
def test_several_chunks(rows, n, d, N, R, only):
    s = _inputs(rows, n, d, N, R, seed=rows + R, only=only)
    x, A, B, scale, base, dC, dx_base = _gpu(s, "x", "A", "B", "scale", "base", "dC", "dx_base")
    off, order = _plan(s, n)
    out, h = gg.lora(x, A, B, off, order, scale=scale, base=base.float(), want_h=True)
    _check_forward(s, out, h, s["scale"], s["base"].float())
    got = gg.lora_backward(dC, x, h, A, B, off, order, scale=scale, dx_base=dx_base)
    _check_backward(s, got, h.cpu(), s["scale"], s["dx_base"])


@pytest.mark.parametrize("rows,n,d,N,R", [(700, 5, 264, 392, 40), (12500, 5, 520, 504, 64)])
def test_what_a_workspace_holds_does_not_show(rows, n, d, N, R):
    s = _inputs(rows, n, d, N, R, seed=11)
    x, A, B, dC = _gpu(s, "x", "A", "B", "dC")
    off, order = _plan(s, n)
    L = gg.lib()
    f = torch.empty(L.moe_lora_workspace_size(rows, n, d, N, R), dtype=torch.uint8, device=DEV)
    b = torch.empty(L.moe_lora_backward_workspace_size(rows, n, d, N, R), dtype=torch.uint8, device=DEV)
    h = torch.randn(rows, R, device=DEV)
    got = []
    for fill in (0, 0x7f, 0xff):   # zeros, large values, NaNs
        f.fill_(fill)
        b.fill_(fill)
        got.append((*gg.lora(x, A, B, off, order, want_h=True, ws=f), *gg.lora_backward(dC, x, h, A, B, off, order, ws=b)))
        assert gg.read_device_status(b) == 0 and (f.numel() == 0 or gg.read_device_status(f) == 0)
    for other in got[1:]:
        assert all(torch.equal(u, v) for u, v in zip(got[0], other))


@pytest.mark.parametrize("rows", [8, 30, 400])
def test_another_adapters_values_stay_its_own(rows):
    # weights, rows and gradients that are not finite reach nothing of another adapter, whichever lies beside it
    n, d, N, R = 3, 136, 72, 24
    s = _inputs(rows, n, d, N, R, seed=12, bare=False)
    row = torch.from_numpy(s["row"]).to(DEV)
    x, A, B, dC = _gpu(s, "x", "A", "B", "dC")
    off, order = _plan(s, n)
    h = torch.randn(rows, R, device=DEV)
    good = (gg.lora(x, A, B, off, order), *gg.lora_backward(dC, x, h, A, B, off, order))
    mine = row == 1
    x[mine], dC[mine], h[mine] = float("nan"), float("inf"), float("nan")
    A[1], B[1] = float("nan"), float("inf")
    bad = (gg.lora(x, A, B, off, order), *gg.lora_backward(dC, x, h, A, B, off, order))
    for g, b, per_row in zip(good, bad, (True, True, False, False)):
        keep = ~mine if per_row else torch.tensor([True, False, True], device=DEV)
        assert torch.equal(g[keep], b[keep]) and not torch.isfinite(b[~keep]).any()


def test_gradients_past_32_bit_offsets():
    rows, N, d, R = 300000, 7168, 8, 8
    dC = torch.zeros(rows, N, dtype=torch.bfloat16, device=DEV)
    dC[-3:] = 1
    x = torch.ones(rows, d, dtype=torch.bfloat16, device=DEV)
    A = torch.ones(1, R, d, dtype=torch.bfloat16, device=DEV)
    B = torch.ones(1, N, R, dtype=torch.bfloat16, device=DEV)
    row = torch.full((rows,), -1, dtype=torch.int32, device=DEV)
    row[-3:] = 0
    off, order = gg.adapter_plan(row, 1)
    dx, dA, dB = gg.lora_backward(dC, x, torch.full((rows, R), 2.0, device=DEV), A, B, off, order, dx_dtype=torch.float32)
    assert (dx[-3:] == N * R).all() and not dx[:-3].any() and (dA == 3 * N).all() and (dB == 6).all()


def _ragged(counts, d, N, R, seed):
    """Rows of each adapter as counted, in a shuffled batch."""
    r = np.random.default_rng(seed)
    s = _inputs(sum(counts), len(counts), d, N, R, seed=seed)
    s["row"] = r.permutation(np.repeat(np.arange(len(counts), dtype=np.int32), counts))
    return s


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_tiles_of_a_row_or_two_over_many_columns(dtype):
    # tiles whose rows one warp brings, or whose base none does, while the stages turn many times: every run the same
    # and none gives up
    counts, d, N, R = [6000, 1, 129, 5, 0, 33], 4104, 2056, 128
    rows, n = sum(counts), len(counts)
    s = _ragged(counts, d, N, R, seed=21)
    x, A, B, base, dC = _gpu(s, "x", "A", "B", "base", "dC")
    off, order = _plan(s, n)
    L = gg.lib()
    assert L.moe_lora_workspace_size(rows, n, d, N, R) > 0
    f = torch.empty(L.moe_lora_workspace_size(rows, n, d, N, R), dtype=torch.uint8, device=DEV)
    b = torch.empty(L.moe_lora_backward_workspace_size(rows, n, d, N, R), dtype=torch.uint8, device=DEV)
    h = torch.randn(rows, R, generator=torch.Generator(DEV).manual_seed(1), device=DEV)
    first = None
    for _ in range(20):
        got = [gg.lora(x, A, B, off, order, out_dtype=dtype, ws=f),
               gg.lora(x, A, B, off, order, base=base.to(dtype), ws=f),
               *gg.lora_backward(dC, x, h, A, B, off, order, dx_dtype=dtype, ws=b),
               gg.lora_backward(dC, x, h, A, B, off, order, dx_dtype=dtype, want_grads=False, ws=b)[0]]
        assert gg.read_device_status(f) == 0 and gg.read_device_status(b) == 0
        first = first or got
        assert all(torch.equal(u, v) for u, v in zip(first, got))
    assert torch.equal(got[2], got[5])
    _check_forward(s, got[0], None, None, None)
    _check_forward(s, got[1], None, None, s["base"].to(dtype))
    _check_backward(s, got[2:5], h.cpu(), None, None)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,n,d,N,R", [(61, 5, 264, 200, 8), (200, 3, 136, 264, 40), (333, 4, 96, 96, 64), (150, 2, 72, 136, 128),
                                          (12500, 5, 520, 504, 64), (6100, 3, 256, 264, 104)])
def test_base_is_added_once(rows, n, d, N, R, dtype):
    """base is no part of the product's sums: beside a base of 2^12 the result is off by its one rounding and, far
    below that, by the product's own bound (_check_forward's, without base in the sums)."""
    s = _inputs(rows, n, d, N, R, seed=R + 1)
    base = (s["base"].float() * 4096).to(dtype)
    if dtype == torch.float32:   # all 24 bits in use
        base += torch.from_numpy(np.random.default_rng(2).uniform(-1, 1, size=base.shape).astype(np.float32))
    x, A, B, scale = _gpu(s, "x", "A", "B", "scale")
    off, order = _plan(s, n)
    out = gg.lora(x, A, B, off, order, scale=scale, base=base.to(DEV))
    want, wh = tuning.lora(s["x"], s["A"], s["B"], s["row"], s["scale"], base)
    mag, magh = tuning.lora(*(np.abs(as_f64(s[v])) for v in ("x", "A", "B")), s["row"], s["scale"].abs())
    tol = np.zeros_like(want)
    for a in range(n):
        r = np.nonzero(s["row"] == a)[0]
        e = depth(d) * magh[r] + (SPLIT + 2.0 ** -23) * np.abs(wh[r]) + depth(2 * R) * np.abs(wh[r])
        tol[r] = abs(float(s["scale"][a])) * (e @ np.abs(as_f64(s["B"][a])).T)
    once = STEP[dtype] + (2.0 ** -24 if dtype == torch.bfloat16 else 0)   # the fp32 sum before a bf16 rounding
    _close(out, want, tol + once * (np.abs(want) + tol), "out")


@pytest.mark.parametrize("rows", [0, 30, 12500])
def test_a_callers_workspace_has_the_calls_status(rows):
    # one workspace for batches of any size: whatever an earlier call left, the status is this call's
    n, d, N, R = 5, 520, 504, 64
    s = _inputs(rows, n, d, N, R, seed=31)
    x, A, B = _gpu(s, "x", "A", "B")
    off, order = _plan(s, n)
    ws = torch.empty(gg.lib().moe_lora_workspace_size(12500, n, d, N, R), dtype=torch.uint8, device=DEV)
    ws.fill_(0xff)
    out = gg.lora(x, A, B, off, order, ws=ws)
    assert gg.read_device_status(ws) == 0
    assert torch.equal(out, gg.lora(x, A, B, off, order))
    if rows < 12500:   # where none is needed, one without room for a status word is left alone
        for short in (ws[:128], ws[64:1024]):
            ws.fill_(0xff)
            gg.lora(x, A, B, off, order, ws=short)
            assert (ws == 0xff).all()


@pytest.mark.parametrize("rows,n,d,N,R,only", [(4000, 1024, 72, 136, 16, [700, 700, 700, 3]), (700, 300, 136, 72, 24, [299]),
                                               (3000, 600, 64, 264, 8, [0, 255, 256, 257, 511, 512, 599]), (2600, 1000, 40, 72, 64, [31, 32])])
def test_few_of_many_held_adapters(rows, n, d, N, R, only):
    # a server holds many adapters, the batch uses a few: several partial sums of some, none of most
    s = _inputs(rows, n, d, N, R, seed=n, only=only)
    x, A, B, scale, dC, dx_base = _gpu(s, "x", "A", "B", "scale", "dC", "dx_base")
    off, order = _plan(s, n)
    out, h = gg.lora(x, A, B, off, order, scale=scale, out_dtype=torch.float32, want_h=True)
    _check_forward(s, out, h, s["scale"], None)
    for dtype in (torch.float32, torch.bfloat16):
        got = gg.lora_backward(dC, x, h, A, B, off, order, scale=scale, dx_base=dx_base, grad_dtype=dtype)
        _check_backward(s, got, h.cpu(), s["scale"], s["dx_base"])
        rest = torch.ones(n, dtype=torch.bool, device=DEV)
        rest[only] = False
        assert not got[1][rest].any() and not got[2][rest].any()


# both sides of the rule that chooses one launch: the same sizes, a row more or less
@pytest.mark.parametrize("rows,n,d,N,R,only", [(12, 3, 136, 72, 32, None), (13, 3, 136, 72, 32, None), (16, 8, 72, 136, 64, None),
                                               (17, 8, 72, 136, 64, None), (96, 24, 64, 264, 40, None), (97, 24, 64, 264, 40, None),
                                               (14, 7, 72, 64, 64, None), (8, 8, 136, 264, 128, None), (9, 8, 136, 264, 128, None),
                                               (130, 130, 136, 264, 104, [0, 0, 5, 129]), (131, 130, 136, 264, 104, [0, 0, 5, 129])])
def test_both_ways_of_few_rows(rows, n, d, N, R, only):
    s = _inputs(rows, n, d, N, R, seed=rows + n, only=only)
    h = torch.from_numpy(np.random.default_rng(7).normal(size=(rows, R)).astype(np.float32))
    dC, x, A, B, scale, base = _gpu(s, "dC", "x", "A", "B", "scale", "dx_base")
    off, order = _plan(s, n)
    for dtype in (torch.float32, torch.bfloat16):
        got = gg.lora_backward(dC, x, h.to(DEV), A, B, off, order, scale=scale, dx_base=base, grad_dtype=dtype)
        _check_backward(s, got, h, s["scale"], s["dx_base"])


def _address(t):
    return None if t is None else t.data_ptr()


@pytest.mark.parametrize("rows,n,d,N,R", [(30, 40, 136, 72, 16), (60, 40, 72, 136, 16), (900, 3, 264, 392, 40), (2600, 2, 136, 264, 24)])
def test_each_result_alone(rows, n, d, N, R):
    # the C call takes any of dx, dA, dB without the others: the same bits, and nothing else is written
    s = _inputs(rows, n, d, N, R, seed=41, only=[0, 0, 0, 1, -1])
    dC, x, A, B, scale, base = _gpu(s, "dC", "x", "A", "B", "scale", "dx_base")
    h = torch.randn(rows, R, generator=torch.Generator(DEV).manual_seed(1), device=DEV)
    off, order = _plan(s, n)
    full = gg.lora_backward(dC, x, h, A, B, off, order, scale=scale, dx_base=base)
    _check_backward(s, full, h.cpu(), s["scale"], s["dx_base"])
    L = gg.lib()
    ws = torch.empty(L.moe_lora_backward_workspace_size(rows, n, d, N, R), dtype=torch.uint8, device=DEV)
    for wanted in range(1, 8):
        got = [torch.full_like(t, 7.0) if wanted >> i & 1 else None for i, t in enumerate(full)]
        ws.fill_(0xff)
        st = L.moe_lora_backward(*map(_address, (dC, x, h, A, B, scale, off, order)), n, rows, d, N, R, _address(base),
                                 _address(got[0]), 2, _address(got[1]), _address(got[2]), 0, ws.data_ptr(), ws.numel(),
                                 torch.cuda.current_stream().cuda_stream)
        assert st == 0 and gg.read_device_status(ws) == 0
        for g, f in zip(got, full):
            assert g is None or torch.equal(g, f), wanted
