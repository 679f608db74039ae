"""Combine's gradient, and the operators in a run as a fine-tuning step uses them: router, balance loss,
experts with adapters beside the down projection, combine, and all the way back."""
import numpy as np
import pytest
import torch

import grouped_gemm_03_b200 as gg
from oracle import as_f64, tuning

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from grouped_gemm_03_b200.build import build
    build()


# dY is one fp32 product rounded to bf16: half a step, 2^-8, and 2^-24 before it.  d_topk_w sums d products,
# d / 32 of one thread in sequence at most (narrow rows take a warp) and a tree of 32 threads and 8 warps.
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d,k,shared", [(1, 8, 1, False), (5, 64, 2, True), (33, 256, 3, False), (64, 264, 4, True),
                                          (20, 1024, 8, True), (9, 1032, 5, False), (130, 2048, 2, False),
                                          (7, 7168, 8, True), (6, 40, 32, True), (11, 328, 9, False)])
def test_combine_backward(T, d, k, shared, dtype):
    r = np.random.default_rng(T)
    rows = T * k + (T if shared else 0)
    Y = torch.from_numpy(r.normal(size=(rows, d))).to(torch.bfloat16)
    dout = torch.from_numpy(r.normal(size=(T, d))).to(dtype)
    t2r = r.permutation(T * k).reshape(T, k).astype(np.int32)
    w = torch.from_numpy(r.random(size=(T, k)).astype(np.float32))
    wY, ww = tuning.combine_backward(dout, Y, t2r, w, T * k if shared else None)
    mag = tuning.combine_backward(dout.abs(), Y.abs(), t2r, w, None)[1]
    args = dout.to(DEV), Y.to(DEV), torch.from_numpy(t2r).to(DEV), w.to(DEV), shared
    dY, dw = gg.combine_backward(*args)
    assert np.all(np.abs(as_f64(dY) - wY) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(wY))
    assert np.all(np.abs(as_f64(dw) - ww) <= (d / 32 + 16) * 2.0 ** -24 * mag)
    assert torch.equal(gg.combine_backward(*args, want_dw=False)[0], dY)
    assert torch.equal(gg.combine_backward(*args, want_dY=False)[1], dw)
    assert torch.equal(gg.combine_backward(args[0], None, *args[2:], want_dw=False)[0], dY)


@pytest.mark.parametrize("shared", [False, True])
def test_combine_backward_of_a_capacity_plan(shared):
    T, d, E, k, cap = 70, 128, 6, 3, 20
    g = torch.Generator().manual_seed(0)
    x = torch.randn(T, d, generator=g).to(torch.bfloat16).to(DEV)
    idx = torch.topk(torch.randn(T, E, generator=g) + torch.arange(E) * 0.5, k, dim=1).indices.to(torch.int32).to(DEV)
    plan = gg.permute(x, idx.contiguous(), E, append_shared=shared, capacity=cap)
    rows = plan["xp"].shape[0]
    kept = int(plan["offsets"][E])
    assert kept < T * k
    Y = torch.randn(rows, d, generator=g).to(torch.bfloat16).to(DEV)
    Y[kept + (T if shared else 0):] = float("nan")      # rows of no token
    w = torch.rand(T, k, generator=g).to(DEV)
    dout = torch.randn(T, d, generator=g).to(torch.bfloat16).to(DEV)
    dout[5] = float("inf")
    dY = torch.full((rows, d), 7.0, dtype=torch.bfloat16, device=DEV)
    _, dw = gg.combine_backward(dout, Y, plan["token_to_row"], w, shared, offsets=plan["offsets"], dY=dY)
    t2r = plan["token_to_row"].cpu().numpy()
    wY, ww = tuning.combine_backward(dout, Y, t2r, w, kept if shared else None)
    live = kept + (T if shared else 0)
    ok = np.isfinite(wY[:live])
    assert np.array_equal(ok, np.isfinite(as_f64(dY)[:live]))
    assert np.all(np.abs(as_f64(dY)[:live] - wY[:live])[ok] <= (2.0 ** -8 + 2.0 ** -23) * np.abs(wY[:live][ok]))
    assert (dY[live:] == 7).all()                       # left as they were
    assert not dw.cpu().numpy()[t2r < 0].any()
    fin = np.isfinite(ww)
    np.testing.assert_allclose(dw.cpu().numpy()[fin], ww[fin], rtol=0, atol=1e-4)
    fresh = gg.combine_backward(dout, Y, plan["token_to_row"], w, shared, offsets=plan["offsets"])[0]
    assert not fresh[live:].any()


def test_a_fine_tuning_step():
    """Gradients of <g, layer(x)> + loss by the router's weights, the adapters and, through autograd in fp64 on the
    host, the same; every library call on the way.  bf16 intermediates (H, Y, dY) bound the agreement: each adds
    2^-8 relative to its own size, a handful of them in a row: 3e-2 of the norm."""
    T, d, E, k, I, n, R = 96, 256, 8, 2, 256, 3, 16
    g = torch.Generator().manual_seed(3)

    def bf(*shape, std=1.0):
        return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16)

    x, W_r = bf(T, d), bf(E, d, std=0.05)
    W1, W2 = bf(E, 2 * I, d, std=0.06), bf(E, d, I, std=0.06)
    A, B = bf(n, R, I, std=0.1), bf(n, d, R, std=0.3)
    scale = torch.tensor([1.0, 0.5, 2.0])
    request = torch.randint(-1, n, (T,), generator=g, dtype=torch.int32)   # the adapter of each token's request
    gout = bf(T, d)
    offsets = torch.tensor([0, 40, 90], dtype=torch.int32)                 # six padded tokens at the end
    alpha = 3.0

    D = lambda *ts: [t.to(DEV) for t in ts]  # noqa: E731
    xg, Wrg, W1g, W2g, Ag, Bg, sg, gg_out, offg = D(x, W_r, W1, W2, A, B, scale, gout, offsets)
    idx, w, logits = gg.router_topk(xg, Wrg, k, want_logits=True)
    loss, counts, prob, coef = gg.balance_loss(logits, idx, alpha, offg)
    plan = gg.permute(xg, idx, E)
    H = gg.grouped_gemm(plan["xp"], W1g, plan["offsets"], I, epilogue=gg.EPI_SILU_GATE)
    Y = gg.grouped_gemm(H, W2g, plan["offsets"], d)
    row = request.to(DEV)[plan["row_to_token"].long()].contiguous()
    aoff, order = gg.adapter_plan(row, n)
    _, h = gg.lora(H, Ag, Bg, aoff, order, scale=sg, base=Y, out=Y, want_h=True)
    out = gg.combine(Y, plan["token_to_row"], w, False, out_dtype=torch.float32)
    dY, dw = gg.combine_backward(gg_out, Y, plan["token_to_row"], w, False)
    dH, dA, dB = gg.lora_backward(dY, H, h, Ag, Bg, aoff, order, scale=sg)
    dlogits = gg.router_backward(logits, idx, dw, counts=counts, coef=coef, seq_offsets=offg)
    dWr = dlogits.double().t() @ xg.double()

    f = torch.float64
    xr, Wr, A64, B64 = x.to(f), W_r.to(f).requires_grad_(), A.to(f).requires_grad_(), B.to(f).requires_grad_()
    p = torch.softmax(xr @ Wr.t(), 1)
    sel = idx.cpu().long()
    wr = torch.gather(p, 1, sel)
    ref = torch.zeros(T, d, dtype=f)
    for j in range(k):
        rows = []
        for t in range(T):
            e, a = int(sel[t, j]), int(request[t])
            u = W1[e].to(f) @ xr[t]
            hid = torch.nn.functional.silu(u[:I]) * u[I:]
            y = W2[e].to(f) @ hid
            if a >= 0:
                y = y + scale[a].to(f) * (B64[a] @ (A64[a] @ hid))
            rows.append(y)
        ref = ref + wr[:, j, None] * torch.stack(rows)
    total = (ref * gout.to(f)).sum()
    bal = 0
    for a, b in ((0, 40), (40, 90)):
        c = torch.zeros(E, dtype=f)
        c.index_add_(0, sel[a:b].flatten(), torch.ones((b - a) * k, dtype=f))
        bal = bal + alpha * E / 2 * (c / (k * (b - a)) * p[a:b].mean(0)).sum()
    (total + bal).backward()

    def near(got, want, tol=3e-2):
        got, want = got.double().cpu(), want.detach()
        assert (got - want).norm() <= tol * want.norm(), float((got - want).norm() / want.norm())

    near(out, ref)
    near(loss, bal.reshape(1), 1e-5)
    near(dWr, Wr.grad)
    near(dA, A64.grad)
    near(dB, B64.grad)
    assert torch.isfinite(dH).all()


@pytest.mark.parametrize("shared", [False, True])
def test_combine_backward_of_slots_without_a_row(shared):
    # a caller's own plan: slots of -1 without the permute's offsets, into a dY that the caller has cleared
    T, d, k = 40, 136, 3
    r = np.random.default_rng(8)
    rows = T * k + (T if shared else 0)
    t2r = r.permutation(T * k).reshape(T, k).astype(np.int32)
    lost = [(0, 0), (3, 2), (7, 0), (7, 1), (7, 2), (39, 1)]
    gone = [int(t2r[at]) for at in lost]
    for at in lost:
        t2r[at] = -1
    Y = torch.from_numpy(r.normal(size=(rows, d))).to(torch.bfloat16)
    Y[gone] = float("nan")
    dout = torch.from_numpy(r.normal(size=(T, d))).to(torch.bfloat16)
    w = torch.from_numpy(r.random(size=(T, k)).astype(np.float32))
    w[3, 2] = float("nan")
    wY, ww = tuning.combine_backward(dout, Y, t2r, w, T * k if shared else None)
    dY = torch.zeros(rows, d, dtype=torch.bfloat16, device=DEV)
    got, dw = gg.combine_backward(dout.to(DEV), Y.to(DEV), torch.from_numpy(t2r).to(DEV), w.to(DEV), shared, dY=dY)
    assert got is dY and not dY[gone].any()
    assert np.all(np.abs(as_f64(dY) - wY) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(wY))
    mag = tuning.combine_backward(dout.abs(), Y.nan_to_num().abs(), t2r, w, None)[1]
    assert np.all(np.abs(as_f64(dw) - ww) <= (d / 32 + 16) * 2.0 ** -24 * mag)


def test_combine_backward_past_32_bit_offsets():
    T, d, k = 40000, 7168, 8                                  # 2.3e9 elements of Y and of dY
    rows = T * k
    t2r = torch.arange(rows, dtype=torch.int32, device=DEV).view(T, k).flip(0).contiguous()
    Y = torch.zeros(rows, d, dtype=torch.bfloat16, device=DEV)
    Y[-k:], Y[:k] = 1, 2
    dout = torch.zeros(T, d, dtype=torch.bfloat16, device=DEV)
    dout[0], dout[-1] = 1, 3
    w = torch.full((T, k), 0.5, device=DEV)
    dY, dw = gg.combine_backward(dout, Y, t2r, w, False)
    assert (dY[-k:] == 0.5).all() and (dY[:k] == 1.5).all() and not dY[k:-k].any()
    assert (dw[0] == d).all() and (dw[-1] == 6 * d).all() and not dw[1:-1].any()


def test_the_experts_input_gradient_with_adapters():
    """dH of Y = H W2^T + s (H A^T) B^T by rows of experts: the frozen weights' part (a product in 32 bits here) goes in
    as dx_base.  dY, dx_base and dH are rounded to bf16, half a step of 2^-8 each: 3 * 2^-8 of the norm at most."""
    T, d, E, k, I, n, R = 80, 264, 4, 2, 136, 3, 24
    g = torch.Generator().manual_seed(5)

    def bf(*shape, std=1.0):
        return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16).to(DEV)

    x, W2, A, B, gout = bf(T, d), bf(E, d, I, std=0.08), bf(n, R, I, std=0.1), bf(n, d, R, std=0.3), bf(T, d)
    scale = torch.tensor([1.0, 0.5, 2.0], device=DEV)
    idx = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int().to(DEV)
    w = torch.rand(T, k, generator=g).to(DEV)
    plan = gg.permute(x, idx, E)
    H, r2t = bf(T * k, I), plan["row_to_token"].long()
    request = torch.randint(-1, n, (T,), generator=g, dtype=torch.int32).to(DEV)
    row = request[r2t].contiguous()
    off, order = gg.adapter_plan(row, n)
    expert = torch.repeat_interleave(torch.arange(E, device=DEV), plan["counts"].long())

    H64 = H.double().requires_grad_()
    a = row.long().clamp(min=0)
    low = torch.einsum("rni,ri->rn", A.double()[a], H64)
    own = torch.einsum("rdn,rn->rd", B.double()[a], low) * (scale[a] * (row >= 0)).double()[:, None]
    Y64 = torch.einsum("rdi,ri->rd", W2.double()[expert], H64) + own
    slot = plan["token_to_row"].long()
    out = (Y64[slot] * w.double()[:, :, None]).sum(1)
    (out * gout.double()).sum().backward()

    Y = Y64.detach().to(torch.bfloat16)
    h = torch.where((row >= 0)[:, None], low, 0.0).detach().float()
    dY, _ = gg.combine_backward(gout, Y, plan["token_to_row"], w, False)
    frozen = torch.einsum("rdi,rd->ri", W2.float()[expert], dY.float()).to(torch.bfloat16)
    dH, dA, dB = gg.lora_backward(dY, H, h, A, B, off, order, scale=scale, dx_base=frozen)
    assert (dH.double() - H64.grad).norm() <= 3 * 2.0 ** -8 * H64.grad.norm()
    assert torch.isfinite(dA).all() and torch.isfinite(dB).all()
