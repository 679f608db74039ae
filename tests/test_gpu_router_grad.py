"""Balance loss and the router's logit gradient against the fp64 oracle.

Tolerances, from the arithmetic: a probability is e^(l-m) / z in fp32 with |l - m| <= 30 here, so its
relative error is at most 30 * 2^-23 (the exponent's argument) + 8 * 2^-24 (exp, sum of z as a tree over
lanes, reciprocal, product) + V * 2^-24 (a lane's own V <= 32 terms) < 6.5e-6 =: EPS.  prob sums positive
terms, at most 64 in sequence and a tree after that: 100 * 2^-24 more.  A gradient row p (G - sum G p) is
then within p * max|G| * (3 EPS + E * 2^-24 for the sum's own additions), plus half a step of its type.
"""
import numpy as np
import pytest
import torch

import grouped_gemm_03_b200 as gg
from oracle import tuning

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 6.5e-6
STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 1e-37, torch.float16: 2.0 ** -25, torch.bfloat16: 1e-37}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from grouped_gemm_03_b200.build import build
    build()


def _inputs(T, E, k, S, dtype, masked, seed=0):
    r = np.random.default_rng(seed)
    logits = torch.from_numpy(r.normal(size=(T, E)) * 2).to(dtype)
    idx = np.argsort(-logits.float().numpy(), axis=1, kind="stable")[:, :k].astype(np.int32)
    used = T - T // 10 if masked else T
    offsets = None if S is None else np.concatenate([[0], np.sort(r.integers(0, used + 1, size=S - 1)), [used]])
    mask = (r.random(T) > 0.2).astype(np.uint8) if masked else None
    return logits, idx, offsets, mask


def _dev(a, dtype=None):
    return None if a is None else torch.as_tensor(a, dtype=dtype).contiguous().to(DEV)


def _check_loss(got, want):
    loss, counts, prob, coef = got
    wl, wc, wp, wk = want
    assert np.array_equal(counts.cpu().numpy(), wc)
    np.testing.assert_allclose(prob.cpu().numpy(), wp, rtol=EPS + 100 * 2 ** -24, atol=1e-30)
    np.testing.assert_allclose(coef.cpu().numpy(), wk, rtol=6 * 2 ** -24, atol=0)
    # products of the three above, positive terms, 64 in sequence at most and a tree
    np.testing.assert_allclose(loss.item(), wl, rtol=EPS + 250 * 2 ** -24, atol=0)


def _check_grad(got, want, p, G, renorm_extra=0.0):
    dt = got.dtype
    got = got.float().cpu().numpy().astype(np.float64)
    E = p.shape[1]
    tol = p * np.abs(G).max(1, keepdims=True) * (1 + renorm_extra) * (3 * EPS + E * 2 ** -24)
    tol = tol + STEP[dt] * np.abs(want) + TINY[dt]
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4], tol[bad][:4])


CASES = [(1, 1, 1, None, torch.float32, False), (1, 8, 2, None, torch.bfloat16, False),
         (7, 5, 5, 3, torch.float32, True), (128, 64, 2, None, torch.float32, False),
         (100, 60, 6, 9, torch.float16, True), (33, 128, 8, 40, torch.bfloat16, True),
         (257, 129, 3, 4, torch.float32, True), (513, 255, 8, 1, torch.bfloat16, False),
         (65, 256, 8, 2, torch.float16, True), (40, 500, 10, 3, torch.float32, False),
         (50, 1000, 32, 5, torch.float32, True), (31, 1024, 32, None, torch.float16, False),
         (20011, 16, 2, 7, torch.float32, True)]


@pytest.mark.parametrize("T,E,k,S,dtype,masked", CASES)
def test_balance_loss(T, E, k, S, dtype, masked):
    logits, idx, offsets, mask = _inputs(T, E, k, S, dtype, masked)
    ws = torch.empty(gg.lib().moe_balance_loss_workspace_size(T, E, S or 1), dtype=torch.uint8, device=DEV)
    got = gg.balance_loss(_dev(logits), _dev(idx), 0.02, _dev(offsets, torch.int32), _dev(mask), ws=ws)
    assert gg.read_device_status(ws) == 0
    _check_loss(got, tuning.balance_loss(logits, idx, 0.02, offsets, mask))


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,E,k,S,dtype,masked", CASES)
def test_router_backward(T, E, k, S, dtype, masked, renorm):
    logits, idx, offsets, mask = _inputs(T, E, k, S, dtype, masked, seed=1)
    r = np.random.default_rng(2)
    g = r.normal(size=(T, k)).astype(np.float32)
    _, counts, _, coef = tuning.balance_loss(logits, idx, 5.0, offsets, mask)
    coef = coef.astype(np.float32)
    dl = np.float32(0.5)
    p = tuning.softmax_rows(logits)
    for parts in ("gates", "balance", "both"):
        gate = g if parts != "balance" else None
        bal = (counts, coef, dl, offsets, mask) if parts != "gates" else None
        for out in (torch.float32, dtype):
            got = gg.router_backward(
                _dev(logits), _dev(idx), _dev(gate), renorm, counts=_dev(counts, torch.int32) if bal else None,
                coef=_dev(coef) if bal else None, d_loss=_dev(np.array([dl])) if bal else None,
                seq_offsets=_dev(offsets, torch.int32), mask=_dev(mask), out_dtype=out)
            want = tuning.router_backward(logits, idx, gate, renorm, bal)
            # |G| at most: the slots' gradients (over the selected mass when renormalised) and the loss's
            G = np.zeros((T, E))
            sel = np.take_along_axis(p, idx, 1).sum(1, keepdims=True) if renorm else 1.0
            if gate is not None:
                G += np.abs(g).max(1, keepdims=True) / sel
            if bal:
                G += np.abs(coef).max() * dl * counts.max()
            _check_grad(got, want, p, G, renorm_extra=1.0 if renorm else 0.0)


def test_what_does_not_count_is_not_read():
    T, E, k = 50, 24, 3
    logits, idx, _, _ = _inputs(T, E, k, None, torch.float32, False, seed=3)
    mask = np.ones(T, np.uint8)
    offsets = np.array([0, 20, 40])
    dead = [3, 21, 39, 41, 49]
    mask[[3, 21, 39]] = 0
    clean = tuning.balance_loss(logits, idx, 1.0, offsets, mask)
    logits[3], logits[21], logits[39, 5], logits[41], logits[49, 0] = (float("nan"), float("inf"), float("nan"),
                                                                       float("nan"), float("-inf"))
    got = gg.balance_loss(_dev(logits), _dev(idx), 1.0, _dev(offsets, torch.int32), _dev(mask))
    _check_loss(got, clean)
    d = gg.router_backward(_dev(logits), _dev(idx), counts=got[1], coef=got[3], seq_offsets=_dev(offsets, torch.int32),
                           mask=_dev(mask))
    assert torch.isfinite(d).all() and not d[dead].any()


def test_minus_infinity_and_lowest_logits():
    T, E, k = 12, 10, 2
    logits = torch.randn(T, E, generator=torch.Generator().manual_seed(0))
    logits[:, 4] = float("-inf")
    logits[2] = float("-inf")             # a row whose mask leaves nothing
    logits[5, 1:] = torch.finfo(torch.float32).min
    logits[6] = torch.finfo(torch.float32).min   # all equal: an even row
    idx = torch.tensor([[0, 1]] * T, dtype=torch.int32)
    g = torch.randn(T, k)
    got = gg.balance_loss(_dev(logits), _dev(idx), 1.0)
    _check_loss(got, tuning.balance_loss(logits, idx, 1.0))
    for renorm in (False, True):
        d = gg.router_backward(_dev(logits), _dev(idx), _dev(g), renorm, counts=got[1], coef=got[3])
        want = tuning.router_backward(logits, idx, g, renorm, (got[1].cpu().numpy(), got[3].cpu().numpy(), 1.0, None, None))
        # row 6 is even over every column, the fifth too: it was written after the -inf
        assert torch.isfinite(d).all() and not d[_dev(logits) == float("-inf")].any()
        np.testing.assert_allclose(d.cpu().numpy(), want, rtol=0, atol=20 * EPS * (1 + np.abs(want).max()))


def test_ids_that_are_none_or_wrong():
    T, E, k = 40, 16, 4
    logits, idx, _, _ = _inputs(T, E, k, None, torch.float32, False, seed=4)
    idx[:, 3] = -1
    ws = torch.empty(gg.lib().moe_balance_loss_workspace_size(T, E, 1), dtype=torch.uint8, device=DEV)
    got = gg.balance_loss(_dev(logits), _dev(idx), 1.0, ws=ws)
    assert gg.read_device_status(ws) == 0
    _check_loss(got, tuning.balance_loss(logits, idx, 1.0))
    g = np.random.default_rng(0).normal(size=(T, k)).astype(np.float32)
    want = tuning.router_backward(logits, idx, g, False)
    idx[7, 0], idx[8, 1] = E, -5
    gg.balance_loss(_dev(logits), _dev(idx), 1.0, ws=ws)
    assert gg.read_device_status(ws) == -1
    d = gg.router_backward(_dev(logits), _dev(idx), _dev(g)).cpu().numpy()
    rows = [t for t in range(T) if t not in (7, 8)]
    np.testing.assert_allclose(d[rows], want[rows], rtol=0, atol=10 * EPS)


def test_the_same_expert_twice_adds_up():
    logits = torch.randn(5, 6, generator=torch.Generator().manual_seed(1))
    idx = np.array([[2, 2, 0]] * 5, np.int32)
    g = np.random.default_rng(1).normal(size=(5, 3)).astype(np.float32)
    for renorm in (False, True):
        d = gg.router_backward(_dev(logits), _dev(idx), _dev(g), renorm).cpu().numpy()
        np.testing.assert_allclose(d, tuning.router_backward(logits, idx, g, renorm), rtol=0, atol=20 * EPS)


def test_one_renormalised_gate_has_no_gradient():
    logits, idx, _, _ = _inputs(64, 32, 1, None, torch.float32, False, seed=6)
    d = gg.router_backward(_dev(logits), _dev(idx), torch.randn(64, 1, device=DEV), True)
    assert not d.any()   # w = p / p is 1 exactly


@pytest.mark.parametrize("offsets", [[1, 4, 8], [0, 5, 3], [0, 4, 9], [0, -2, 8]])
def test_bad_offsets_are_reported(offsets):
    # every read stays inside the tokens: the kernel holds a segment to its chunk and T
    logits, idx, _, _ = _inputs(8, 4, 1, None, torch.float32, False)
    ws = torch.empty(gg.lib().moe_balance_loss_workspace_size(8, 4, 2), dtype=torch.uint8, device=DEV)
    gg.balance_loss(_dev(logits), _dev(idx), 1.0, _dev(np.array(offsets), torch.int32), ws=ws)
    assert gg.read_device_status(ws) == -5


def test_no_tokens():
    e = torch.empty
    loss, counts, prob, coef = gg.balance_loss(e(0, 8, device=DEV), e(0, 2, dtype=torch.int32, device=DEV), 1.0)
    assert loss.item() == 0 and not counts.any() and not prob.any() and not coef.any()
    d = gg.router_backward(e(0, 8, device=DEV), e(0, 2, dtype=torch.int32, device=DEV), e(0, 2, device=DEV))
    assert d.shape == (0, 8)


def test_in_place_gradient():
    logits, idx, _, _ = _inputs(77, 40, 4, None, torch.float32, False, seed=8)
    g = torch.randn(77, 4, device=DEV)
    l = _dev(logits)
    want = gg.router_backward(l, _dev(idx), g)
    gg.router_backward(l, _dev(idx), g, out=l)
    assert torch.equal(l, want)


def test_captured_on_a_side_stream_and_replayed():
    T, E, k = 300, 64, 4
    logits, idx, offsets, mask = _inputs(T, E, k, 5, torch.float32, True, seed=9)
    l, i, o, m = _dev(logits), _dev(idx), _dev(offsets, torch.int32), _dev(mask)
    g = torch.randn(T, k, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    gg.router_backward(l, i, g, stream=side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        loss, counts, prob, coef = gg.balance_loss(l, i, 0.1, o, m)
        d = gg.router_backward(l, i, g, counts=counts, coef=coef, seq_offsets=o, mask=m)
    for seed in (10, 11):
        fresh, idx2, _, _ = _inputs(T, E, k, 5, torch.float32, True, seed=seed)
        l.copy_(fresh)
        i.copy_(torch.from_numpy(idx2))
        graph.replay()
        torch.cuda.synchronize()
        eager = gg.balance_loss(l, i, 0.1, o, m)
        for a, b in zip((loss, counts, prob, coef), eager):
            assert torch.equal(a, b)
        assert torch.equal(d, gg.router_backward(l, i, g, counts=eager[1], coef=eager[3], seq_offsets=o, mask=m))
        _check_loss(eager, tuning.balance_loss(fresh, idx2, 0.1, offsets, mask))


# many short sequences, more of them than a block has threads, slots past eight, chunks past a block's threads
@pytest.mark.parametrize("T,E,k,S,dtype", [(3000, 96, 9, 400, torch.bfloat16), (600, 1000, 32, 590, torch.float32),
                                           (120000, 8, 2, 300, torch.float16), (130001, 24, 1, None, torch.bfloat16),
                                           (2000, 7, 3, 2, torch.float32)])
def test_balance_loss_of_large_batches(T, E, k, S, dtype):
    logits, idx, offsets, mask = _inputs(T, E, k, S, dtype, True, seed=12)
    ws = torch.empty(gg.lib().moe_balance_loss_workspace_size(T, E, S or 1), dtype=torch.uint8, device=DEV)
    args = _dev(logits), _dev(idx), 0.5, _dev(offsets, torch.int32), _dev(mask)
    ws.fill_(0xff)
    got = gg.balance_loss(*args, ws=ws)
    assert gg.read_device_status(ws) == 0
    _check_loss(got, tuning.balance_loss(logits, idx, 0.5, offsets, mask))
    for a, b in zip(got, gg.balance_loss(*args)):   # bit for bit, whatever the workspace held
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_rows_of_the_types_lowest_value(dtype):
    T, E, k = 40, 24, 3
    logits = torch.randn(T, E, generator=torch.Generator().manual_seed(2)).to(dtype)
    low = torch.finfo(dtype).min
    logits[3] = low                       # all equal: an even row
    logits[4, 1:] = low
    logits[5] = float("-inf")
    logits[6, :20] = float("-inf")
    logits[6, 20:] = low                  # even over the last four
    logits[7] = torch.finfo(dtype).max    # even, too
    idx = torch.tensor([[0, 21, 22]] * T, dtype=torch.int32)
    g = torch.randn(T, k)
    got = gg.balance_loss(_dev(logits), _dev(idx), 1.0)
    _check_loss(got, tuning.balance_loss(logits, idx, 1.0))
    d = gg.router_backward(_dev(logits), _dev(idx), _dev(g), counts=got[1], coef=got[3])
    want = tuning.router_backward(logits, idx, g, False, (got[1].cpu().numpy(), got[3].cpu().numpy(), 1.0, None, None))
    np.testing.assert_allclose(d.cpu().numpy(), want, rtol=0, atol=20 * EPS * (1 + np.abs(want).max()))


def _large_rows(T, E, dtype, seed):
    """Finite rows whose maximum is far from 0, between the types' borders, among ordinary ones."""
    l = torch.randn(T, E, generator=torch.Generator().manual_seed(seed))
    at = 1
    for m in (1e6, 2.0 ** 20 - 1, 2.0 ** 20 + 1, 3e7, 1e9, 1e10, 1e12, 1e15, 1e20, 1e29, 1e31):
        for v in (m, -m):
            l[at] = v                                     # all equal: an even row
            l[at + 1] = v
            l[at + 1, 1::2] = -1e35                       # even over half of them
            l[at + 2, 1:], l[at + 2, 0] = v, 2 * abs(v)   # one takes all
            l[at + 3] = v + torch.arange(E) % 7 * 0.5     # as far apart as the type holds there
            at += 5                                       # an ordinary row between
    return l.to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E", [(120, 24), (700, 128), (120, 999), (600, 1024)])
def test_large_finite_rows(T, E, dtype):
    """The exponent's argument is (l - m) log2 e in fp32 there too, so the tolerances of ordinary rows hold."""
    k = 3
    logits = _large_rows(T, E, dtype, seed=E)
    idx = np.argsort(-logits.float().numpy(), axis=1, kind="stable")[:, :k].astype(np.int32)
    idx[::2, 2] = E - 1
    offsets = np.array([0, T // 3, T])
    got = gg.balance_loss(_dev(logits), _dev(idx), 1.0, _dev(offsets, torch.int32))
    _check_loss(got, tuning.balance_loss(logits, idx, 1.0, offsets))
    p = tuning.softmax_rows(logits)
    g = np.random.default_rng(3).normal(size=(T, k)).astype(np.float32)
    counts, coef = got[1].cpu().numpy(), got[3].cpu().numpy()
    for renorm in (False, True):
        d = gg.router_backward(_dev(logits), _dev(idx), _dev(g), renorm, counts=got[1], coef=got[3],
                               seq_offsets=_dev(offsets, torch.int32))
        want = tuning.router_backward(logits, idx, g, renorm, (counts, coef, 1.0, offsets, None))
        sel = np.take_along_axis(p, idx, 1).sum(1, keepdims=True) if renorm else 1.0
        G = np.abs(g).max(1, keepdims=True) / sel + coef.max() * counts.max()
        _check_grad(d, want, p, G, renorm_extra=1.0 if renorm else 0.0)


@pytest.mark.parametrize("offsets,status", [([0, 0, 0], 0), ([0, 0, 5], -5), ([0, -1, 0], -5), ([2, 0, 0], -5), ([0, 3, 0], -5)])
def test_offsets_of_no_tokens(offsets, status):
    e = torch.empty
    ws = e(gg.lib().moe_balance_loss_workspace_size(0, 8, 2), dtype=torch.uint8, device=DEV)
    ws.fill_(0xff)
    loss, counts, prob, coef = gg.balance_loss(e(0, 8, device=DEV), e(0, 2, dtype=torch.int32, device=DEV), 1.0,
                                               _dev(np.array(offsets), torch.int32), ws=ws)
    assert gg.read_device_status(ws) == status
    assert loss.item() == 0 and not counts.any() and not prob.any() and not coef.any()


@pytest.mark.parametrize("renorm", [False, True])
def test_a_mask_is_the_losss_alone(renorm):
    # without the loss's counts, mask and offsets change nothing; with them, the gates' part of a masked token stays
    T, E, k = 90, 40, 4
    logits, idx, offsets, mask = _inputs(T, E, k, 3, torch.float32, True, seed=13)
    g = torch.randn(T, k, generator=torch.Generator().manual_seed(4)).to(DEV)
    args = _dev(logits), _dev(idx), g, renorm
    plain = gg.router_backward(*args)
    assert torch.equal(plain, gg.router_backward(*args, mask=_dev(mask), seq_offsets=_dev(offsets, torch.int32)))
    _, counts, _, coef = gg.balance_loss(_dev(logits), _dev(idx), 1.0, _dev(offsets, torch.int32), _dev(mask))
    both = gg.router_backward(*args, counts=counts, coef=coef, mask=_dev(mask), seq_offsets=_dev(offsets, torch.int32))
    dead = torch.from_numpy(mask == 0).to(DEV)
    dead[int(offsets[-1]):] = True
    assert torch.equal(both[dead], plain[dead]) and not torch.equal(both, plain)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,k", [(16, 2), (24, 5), (256, 4), (96, 32), (1000, 8)])
def test_renormalised_gates_far_below_the_row(E, k, dtype):
    """Ids that something else than these logits chose: the selected experts' probabilities underflow in fp32, their
    softmax among themselves does not.  w (g - sum w g) is then within a few EPS of max|g| (1 at most here)."""
    T = 65
    r = np.random.default_rng(E)
    logits = torch.from_numpy(r.normal(size=(T, E))).to(dtype)
    idx = np.stack([r.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    for t in range(0, T, 2):
        logits[t, idx[t].astype(np.int64)] += (-40, -95, -130, -600)[t // 2 % 4]
    idx[6, 1] = -1                                        # a slot without an expert
    logits[8, int(idx[8, 0])] = float("-inf")             # one of the selected has none of the mass
    logits[10, torch.from_numpy(idx[10]).long()] = float("-inf")   # nor has any
    g = r.uniform(-1, 1, size=(T, k)).astype(np.float32)
    got = gg.router_backward(_dev(logits), _dev(idx), _dev(g), True).cpu().numpy()
    want = tuning.router_backward(logits, idx, g, True)
    np.testing.assert_allclose(got, want, rtol=0, atol=20 * EPS)
    assert (np.abs(want).max(1) > 1e-3).sum() >= T - 4   # of two slots, rows 6 and 8 keep one: no gradient, as row 10


@pytest.mark.parametrize("T,E,k,S", [(300, 24, 3, 5000), (1, 8, 2, 700), (900, 40, 2, 20000), (512, 1024, 8, 300)])
def test_more_sequences_than_tokens(T, E, k, S):
    logits, idx, offsets, mask = _inputs(T, E, k, S, torch.float32, T > 1, seed=S)
    args = _dev(logits), _dev(idx), 0.5, _dev(offsets, torch.int32), _dev(mask)
    got = gg.balance_loss(*args)
    _check_loss(got, tuning.balance_loss(logits, idx, 0.5, offsets, mask))
    bare = gg.balance_loss(*args, want_prob=False)
    assert bare[2] is None and all(torch.equal(a, b) for a, b in zip(got, bare) if b is not None)
    d = gg.router_backward(args[0], args[1], counts=got[1], coef=got[3], seq_offsets=args[3], mask=args[4])
    bal = (got[1].cpu().numpy(), got[3].cpu().numpy(), 1.0, offsets, mask)
    want = tuning.router_backward(logits, idx, balance=bal)
    G = np.full((T, E), float((got[3][:, None] * got[1]).max()))
    _check_grad(d, want, tuning.softmax_rows(logits), G)


def test_logits_past_32_bit_offsets():
    T, E, k, last = 2200000, 1024, 2, 100
    logits = torch.zeros(T, E, dtype=torch.bfloat16, device=DEV)   # 2^31 elements before the last rows
    logits[-last:].normal_(0, 2, generator=torch.Generator(DEV).manual_seed(1))
    idx = torch.zeros(T, k, dtype=torch.int32, device=DEV)
    idx[-last:] = torch.topk(logits[-last:].float(), k, dim=1).indices.int()
    d_w = torch.zeros(T, k, device=DEV)
    d_w[-last:].normal_(generator=torch.Generator(DEV).manual_seed(2))
    offsets = torch.tensor([0, T - last, T], dtype=torch.int32, device=DEV)
    loss, counts, prob, coef = gg.balance_loss(logits, idx, 0.5, offsets)
    end = logits[-last:].contiguous(), idx[-last:].contiguous()
    _, c1, p1, _ = gg.balance_loss(*end, 0.5)
    assert torch.equal(counts[1:], c1) and int(counts[0, 0]) == (T - last) * k and not counts[0, 1:].any()
    assert torch.allclose(prob[1:], p1, rtol=EPS, atol=0)
    # equal logits: 1 / E each, summed over 2.2 million rows in chains of T / (2 * 148 * 8) and a tree behind them
    assert torch.allclose(prob[0], torch.full((E,), 1 / E, device=DEV), rtol=T / (2 * 148 * 8) * 2 ** -24 + EPS, atol=0)
    for renorm in (False, True):
        d = gg.router_backward(logits, idx, d_w, renorm, out_dtype=torch.bfloat16)
        assert torch.equal(d[-last:], gg.router_backward(*end, d_w[-last:].contiguous(), renorm, out_dtype=torch.bfloat16))
        assert not d[:-last].any()
