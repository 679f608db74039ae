"""How exact the adapters' fp32 results are, as a norm: what element-wise bounds leave room for.

A sum of s tensor-core steps cuts each partial sum p off at 24 bits: half a unit on average, 0.72 * 2^-24 |p| over
a binade, always towards 0.  Of sums of independent terms the i-th partial one holds i / s of the result, so the
steps together leave 0.36 s 2^-24 of the result's norm; roundings to nearest (joins, the last rounding) leave 2^-23
beside that.  h and dh enter their products as three bf16 terms, all of an fp32 value, the smaller ones first: only
the largest's steps cut a whole sum off.  Two terms would leave the rounding of the second, 2.4e-6 of a normal value:
where chains are short, the tests show on their oracle that the bounds tell that apart.
"""
import pytest
import torch

import grouped_gemm_03_b200 as gg

pytestmark = pytest.mark.gpu
DEV = "cuda"


def bound(steps):
    return 0.36 * steps * 2.0 ** -24 + 2.0 ** -23


def _off(got, want):
    return float((got.double() - want).norm() / want.norm())


def _two_terms(v):
    hi = v.to(torch.bfloat16)
    return (hi.double() + (v - hi.float()).to(torch.bfloat16).double())


@pytest.fixture(scope="module", autouse=True)
def _built():
    from grouped_gemm_03_b200.build import build
    build()


def _batch(rows, n, d, N, R, seed):
    g = torch.Generator(DEV).manual_seed(seed)

    def bf(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=DEV) * std).to(torch.bfloat16)

    row = torch.arange(rows, device=DEV, dtype=torch.int32) % n
    s = dict(row=row, x=bf(rows, d), A=bf(n, R, d, std=d ** -0.5), B=bf(n, N, R, std=0.2), dC=bf(rows, N),
             h=torch.randn(rows, R, generator=g, device=DEV), scale=torch.rand(n, generator=g, device=DEV) + 0.5)
    return s, gg.adapter_plan(row, n)


def _rows_of(s):
    return [(s["row"] == a).nonzero().flatten() for a in range(len(s["A"]))]


# one launch: the longest chain is a warp's columns of x (d / 128 steps and fewer) and R / 16 of the largest term; two
# launches: d / 16 steps over up to four accumulators of whole blocks of 128 columns (eight up to rank 32)
@pytest.mark.parametrize("rows,n,d,N,R,launches,steps,steps_h", [
    (61, 5, 512, 704, 64, 1, 8, 4), (100, 3, 264, 136, 128, 1, 11, 3), (300, 4, 1032, 512, 24, 1, 11, 9), (90, 2, 512, 264, 8, 1, 5, 4),
    (20000, 5, 264, 504, 64, 2, 12, 8), (80000, 1, 520, 1000, 16, 2, 9, 8), (6100, 3, 256, 264, 104, 2, 16, 8)])
def test_forward(rows, n, d, N, R, launches, steps, steps_h):
    s, (off, order) = _batch(rows, n, d, N, R, seed=rows)
    assert (gg.lib().moe_lora_workspace_size(rows, n, d, N, R) > 0) == (launches == 2)
    out, h = gg.lora(s["x"], s["A"], s["B"], off, order, scale=s["scale"], out_dtype=torch.float32, want_h=True)
    wh, want, less = (torch.zeros(rows, v, dtype=torch.float64, device=DEV) for v in (R, N, N))
    for a, r in enumerate(_rows_of(s)):
        wh[r] = s["x"][r].double() @ s["A"][a].double().t()
        b = s["B"][a].double().t()
        sc = s["scale"][a]
        want[r] = sc.double() * wh[r] @ b
        less[r] = _two_terms((wh[r] * sc.double()).float()) @ b
    assert _off(h, wh) <= bound(steps_h)
    assert _off(out, want) <= bound(steps) < _off(less, want)


def test_projection_of_wide_rows():
    # two slices of 28 blocks over eight accumulators: four blocks, 32 steps; all into one would be 224
    rows, n, d, N, R = 8192, 8, 7168, 64, 32
    s, (off, order) = _batch(rows, n, d, N, R, seed=1)
    h = gg.lora(s["x"], s["A"], s["B"], off, order, want_h=True)[1]
    want = torch.zeros(rows, R, dtype=torch.float64, device=DEV)
    for a, r in enumerate(_rows_of(s)):
        want[r] = s["x"][r].double() @ s["A"][a].double().t()
    assert _off(h, want) <= bound(32)


def _gradients(s, scale, terms=lambda v: v.double()):
    """(dx, dA, dB) in 64 bits, dh and s h as `terms` of them."""
    dx = torch.zeros(s["x"].shape, dtype=torch.float64, device=DEV)
    dA, dB = (torch.zeros(s[v].shape, dtype=torch.float64, device=DEV) for v in ("A", "B"))
    for a, r in enumerate(_rows_of(s)):
        dc, sc = s["dC"][r].double(), scale[a].double()
        dh = terms((sc * dc @ s["B"][a].double()).float()) if terms is _two_terms else sc * dc @ s["B"][a].double()
        dx[r] = dh @ s["A"][a].double()
        dA[a] = dh.t() @ s["x"][r].double()
        dB[a] = dc.t() @ (terms(s["h"][r] * scale[a]) if terms is _two_terms else s["h"][r].double() * sc)
    return dx, dA, dB


# dh: N / 16 steps; then 8 steps to 128 rows of an adapter (dA, dB) or R / 16 of the largest term (dx)
@pytest.mark.parametrize("rows,n,d,N,R", [(800, 8, 264, 128, 64), (1000, 8, 136, 128, 16), (510, 4, 520, 72, 32)])
def test_gradients(rows, n, d, N, R):
    s, (off, order) = _batch(rows, n, d, N, R, seed=R)
    got = gg.lora_backward(s["dC"], s["x"], s["h"], s["A"], s["B"], off, order, scale=s["scale"], dx_dtype=torch.float32)
    want, less = _gradients(s, s["scale"]), _gradients(s, s["scale"], _two_terms)
    of_dh = (N + 15) // 16
    for g, w, l, steps in zip(got, want, less, (of_dh + (R + 15) // 16, of_dh + 8, 8)):
        assert _off(g, w) <= bound(steps) < _off(l, w)


def test_gradients_of_many_rows():
    # a sum ends after 1024 rows, 64 steps; 4096 in one would be 256
    s, (off, order) = _batch(4096, 1, 264, 128, 16, seed=2)
    got = gg.lora_backward(s["dC"], s["x"], s["h"], s["A"], s["B"], off, order, scale=s["scale"], dx_dtype=torch.float32)
    for g, w, steps in zip(got, _gradients(s, s["scale"]), (8 + 1, 8 + 64, 64)):
        assert _off(g, w) <= bound(steps)


def test_gradients_of_many_rows_at_a_high_rank():
    # above rank 64 the three terms take turns in one accumulator: three times the steps
    s, (off, order) = _batch(3000, 2, 264, 128, 128, seed=4)
    got = gg.lora_backward(s["dC"], s["x"], s["h"], s["A"], s["B"], off, order, scale=s["scale"], dx_dtype=torch.float32)
    for g, w, steps in zip(got, _gradients(s, s["scale"]), (8 + 8, 8 + 3 * 64, 3 * 64)):
        assert _off(g, w) <= bound(steps)


@pytest.mark.parametrize("rows,n,R", [(12, 8, 64), (60, 100, 128), (40, 10, 16)])
def test_gradients_of_few_rows(rows, n, R):
    # fp32 multiply-adds, rounded to nearest: N = 1032 columns in chains of up to 33, then sums over lanes, warps and CTAs
    s, (off, order) = _batch(rows, n, 264, 1032, R, seed=3)
    got = gg.lora_backward(s["dC"], s["x"], s["h"], s["A"], s["B"], off, order, scale=s["scale"], dx_dtype=torch.float32)
    for g, w in zip(got, _gradients(s, s["scale"])):
        assert _off(g, w) <= 6 * 2.0 ** -24   # a random walk of 33 half steps, 2^-24 each, and the sums behind it
