"""GPU tests of routing by scores and of its gradient against 64-bit definitions: ids exactly, weights and
gradients within bounds counted in roundings."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import quantized_mixture_experts_route_amd as qm
from tests import _fp8_ref as ref

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")


def _check(logits, bias, k, score, groups=1, kept=None, best=1, normalize=True, scale=1.0):
    kept = groups if kept is None else kept
    sigmoid = score == qm.SCORE_SIGMOID
    ids, w = qm.route_scores(logits, k, score=score, bias=bias, n_groups=groups, top_groups=kept, group_top=best,
                             normalize=normalize, scale=scale)
    assert ids.dtype == torch.int32 and w.dtype == F32 and ids.shape == w.shape == (logits.shape[0], k)
    x = logits.float().cpu().numpy()
    b = None if bias is None else bias.cpu().numpy()
    ids, w = ids.cpu().numpy(), w.cpu().numpy()
    for t in range(len(x)):
        want = ref.choose(x[t], b, k, sigmoid, groups, kept, best)
        assert np.array_equal(ids[t], want), (t, ids[t], want)
        wants = ref.weights(x[t], want, sigmoid, normalize, scale)
        tol = ref.weight_error(x[t], want, x.shape[1]) * ref.U32 * np.abs(wants) + abs(scale) * 2.0 ** -125
        assert np.all(np.abs(w[t] - wants) <= tol), (t, w[t], wants)
    return torch.from_numpy(ids), torch.from_numpy(w)


# T, E, k, groups, kept, best
SIZES = [(1, 1, 1, 1, 1, 1), (1, 2, 2, 1, 1, 1), (3, 7, 3, 1, 1, 1), (5, 60, 4, 1, 1, 1), (4, 64, 64, 1, 1, 1),
         (33, 65, 6, 1, 1, 1), (2, 128, 8, 8, 4, 2), (130, 256, 8, 8, 4, 2), (17, 256, 8, 8, 1, 1), (6, 512, 10, 1, 1, 1),
         (9, 513, 10, 27, 3, 2), (3, 1024, 16, 64, 5, 2), (2, 1023, 64, 3, 2, 1), (40, 160, 6, 8, 3, 1),
         (12, 64, 3, 64, 3, 2), (300, 8, 2, 1, 1, 1), (70, 16, 4, 4, 2, 2)]


@pytest.mark.parametrize("score", [qm.SCORE_SOFTMAX, qm.SCORE_SIGMOID])
@pytest.mark.parametrize("T,E,k,groups,kept,best", SIZES)
def test_choice_and_weights(T, E, k, groups, kept, best, score):
    g = torch.Generator(device="cuda").manual_seed(T * E)
    for dtype, biased, normalize in ((F32, True, True), (BF16, True, False), (F16, False, True), (F32, False, False)):
        logits = (torch.randn(T, E, generator=g, device="cuda") * 2).to(dtype)
        bias = torch.randn(E, generator=g, device="cuda") * 0.2 if biased else None
        _check(logits, bias, k, score, groups, kept, best, normalize, 2.5 if biased else 1.0)


@pytest.mark.parametrize("score", [qm.SCORE_SOFTMAX, qm.SCORE_SIGMOID])
def test_ties_go_to_the_lower_index(score):
    # few different logits (and, without a bias, few different choices): ties at every border
    g = torch.Generator(device="cuda").manual_seed(5)
    logits = torch.randint(-2, 3, (64, 96), generator=g, device="cuda").to(F16) / 2
    logits[0] = 0.0
    logits[1, ::2] = -0.0
    logits[1, 1::2] = 0.0
    for bias in (None, torch.zeros(96, device="cuda"), torch.randint(0, 2, (96,), generator=g, device="cuda").float()):
        ids, _ = _check(logits, bias, 7, score)
        _check(logits, bias, 7, score, 8, 3, 2)
        _check(logits, bias, 7, score, 8, 3, 1)
    assert qm.route_scores(logits[:2], 7, score=score)[0].cpu().tolist() == [list(range(7))] * 2


@pytest.mark.parametrize("score", [qm.SCORE_SOFTMAX, qm.SCORE_SIGMOID])
def test_choices_that_float32_does_not_tell_apart(score):
    # the bias makes up for the scores' differences up to a few units of float64's tenth digit
    T, E = 40, 64
    rng = np.random.default_rng(9)
    logits = rng.normal(size=(T, E)).astype(np.float32)
    logits[:] = logits[0]
    s = ref.scores(logits[0], score == qm.SCORE_SIGMOID)
    base = (s.max() + 0.25 - s).astype(np.float32)  # s + base is 1 in 2^24 around one value
    for seed in range(4):
        bias = torch.from_numpy(base * np.float32(1 + seed * 2.0 ** -20)).cuda()
        _check(torch.from_numpy(logits[:4]).cuda(), bias, 12, score)
        _check(torch.from_numpy(logits[:4]).cuda(), bias, 12, score, 8, 4, 2)


@pytest.mark.parametrize("score", [qm.SCORE_SOFTMAX, qm.SCORE_SIGMOID])
@pytest.mark.parametrize("E,k", [(48, 6), (64, 40), (256, 8), (1024, 20)])
def test_chains_of_choices_next_to_one_another(score, E, k):
    # neighbours a unit or a few of float32 apart: shorter and longer than the slots, across the last slot and
    # through every expert, up and down, on top of one another and far below the row's largest
    near = 1 + torch.arange(E, dtype=torch.float64).mul(2.0 ** -22)
    rows = [near, near.flip(0), -near, near.mul(-70), near.mul(0.25).where(torch.arange(E) % 3 > 0, torch.tensor(-5.0).double())]
    logits = torch.stack(rows).float()
    logits = torch.cat((logits, logits[:, torch.randperm(E, generator=torch.Generator().manual_seed(E))]))
    spread = torch.randn(2, E, generator=torch.Generator().manual_seed(1))
    spread[0, 5:5 + k - 1] = 4.0 + torch.arange(k - 1) * 2.0 ** -21   # ends before the last slot
    spread[1, 5:5 + k + 2] = 4.0 - torch.arange(k + 2) * 2.0 ** -21   # ends behind it
    top = torch.cat((logits, spread))
    top[3] -= 1.0
    top[3, E // 2] = 20.0  # scores around exp(-90): below float32's normal range
    for bias in (None, torch.zeros(E), torch.full((E,), 3.0)):
        b = None if bias is None else bias.cuda()
        _check(top.cuda(), b, k, score)
        _check(top.cuda(), b, k, score, 8, 5, 2)
        _check(top.cuda(), b, k, score, 8, 5, 1)


@pytest.mark.parametrize("score", [qm.SCORE_SOFTMAX, qm.SCORE_SIGMOID])
def test_biases_far_larger_than_the_scores(score):
    # a group's rank is the sum of a large and a small choice: its error goes with them, not with the sum
    g = torch.Generator().manual_seed(12)
    logits = torch.randn(50, 64, generator=g)
    for large in (3.0, 100.0, 1e6, 1e30):
        bias = torch.full((64,), -large)
        bias[::8] = large
        _check(logits.cuda(), bias.cuda(), 12, score, 8, 4, 2)
        _check(logits.cuda(), bias.cuda(), 12, score)
    bias[3] = INF
    bias[4] = -INF
    _check(logits.cuda(), bias.cuda(), 12, score, 8, 4, 2)


@pytest.mark.parametrize("score", [qm.SCORE_SOFTMAX, qm.SCORE_SIGMOID])
def test_ranks_that_leave_the_range_of_float32(score):
    # two finite choices that add up to more, or less, than float32 holds; -inf is a group without experts
    low = torch.finfo(F32).min
    g = torch.Generator().manual_seed(8)
    bias = torch.tensor([0.0] * 4 + [-1.8e38, -1.8e38, -3.3e38, -3.3e38] + [-2e38] * 4)
    _check(torch.randn(9, 12, generator=g).cuda(), bias.cuda(), 8, score, 3, 2, 2)
    for E, groups, kept, k in ((64, 8, 5, 24), (256, 8, 4, 60), (160, 8, 4, 30), (1024, 64, 20, 64), (48, 8, 3, 16)):
        size, logits = E // groups, torch.randn(12, E, generator=g)
        logits[3, :size] = logits[4, size:] = -INF
        for named in ([0.0, low], [0.0, low, -3e38, -2e38, -1.8e38], [1.8e38, 2e38, -low, low, 0.0], [low]):
            by_group = torch.tensor(named)[torch.randint(0, len(named), (groups, 1), generator=g)]
            by_expert = torch.tensor(named)[torch.randint(0, len(named), (E,), generator=g)]
            for bias in (by_group.expand(groups, size).reshape(E), by_expert):
                for best in (1, 2):
                    _check(logits.cuda(), bias.cuda(), k, score, groups, kept, best)


@pytest.mark.parametrize("score", [qm.SCORE_SOFTMAX, qm.SCORE_SIGMOID])
@pytest.mark.parametrize("normalize", [True, False])
def test_masked_experts_and_rows(score, normalize):
    g = torch.Generator(device="cuda").manual_seed(3)
    logits = torch.randn(40, 48, generator=g, device="cuda")
    logits[torch.rand(40, 48, generator=g, device="cuda") < 0.6] = -INF
    logits[0] = -INF                      # nothing left
    logits[1] = -INF
    logits[1, 47] = -3.0                  # one expert left
    logits[2, 5:] = torch.finfo(F32).min  # the type's lowest value is a value
    logits[3] = torch.finfo(F32).min
    logits[4, :24] = -INF                 # groups without experts
    bias = torch.randn(48, generator=g, device="cuda")
    for b in (None, bias):
        ids, w = _check(logits, b, 6, score, normalize=normalize)
        assert ids[0].eq(-1).all() and w[0].eq(0).all()
        assert ids[1].tolist() == [47] + [-1] * 5
        _check(logits, b, 6, score, 8, 3, 2, normalize)
        _check(logits, b, 6, score, 8, 3, 1, normalize)
    bias[10] = -INF  # an expert taken out by its bias
    ids, _ = _check(logits, bias, 30, score, normalize=normalize)
    assert not ids.eq(10).any()


def test_sigmoid_weights_of_scores_below_float32():
    logits = torch.tensor([[-200.0, -201.0, -300.0, -90.0], [-1e30, -1e30, -2e30, -3e30], [100.0, 200.0, 88.0, -88.0],
                           [0.0, -104.0, -150.0, 30.0]], device="cuda")
    _check(logits, None, 3, qm.SCORE_SIGMOID)
    _check(logits[2:], None, 3, qm.SCORE_SIGMOID, normalize=False)
    _check(logits, None, 3, qm.SCORE_SOFTMAX)


def test_nan_and_infinities():
    x = torch.randn(6, 20, device="cuda")
    x[0, 7] = NAN
    x[1, 3] = INF
    x[2, :] = NAN
    ids, w = qm.route_scores(x, 4, score=qm.SCORE_SIGMOID)
    assert ids[0, 0] == 7 and w[0].isnan().all()            # chosen first, and in the sum
    assert ids[1, 0] == 3 and w[1].isfinite().all()
    assert ids[2].tolist() == [0, 1, 2, 3] and w[2].isnan().all()
    _, w = qm.route_scores(x, 4, score=qm.SCORE_SIGMOID, normalize=False)
    assert w[0, 0].isnan() and w[0, 1:].isfinite().all()
    for bias in (None, torch.randn(20, device="cuda")):
        for normalize in (True, False):
            ids, w = qm.route_scores(x, 4, bias=bias, normalize=normalize)
            assert w[:3].isnan().all() and w[3:].isfinite().all()
            for row in ids.tolist():
                assert len(set(row)) == 4 and all(0 <= e < 20 for e in row)


@pytest.mark.parametrize("score", [qm.SCORE_SOFTMAX, qm.SCORE_SIGMOID])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("T,E,k,dtype", [(1, 1, 1, F32), (3, 5, 2, F16), (40, 60, 4, BF16), (9, 256, 8, F32), (2, 1024, 64, F32),
                                         (65, 513, 10, BF16), (130, 64, 6, F16), (7, 128, 1, F32), (33, 8, 8, BF16)])
def test_gradient(T, E, k, dtype, score, normalize):
    g = torch.Generator(device="cuda").manual_seed(T + E)
    logits = (torch.randn(T, E, generator=g, device="cuda") * 2).to(dtype)
    if T > 2:
        logits[1] = -INF
        logits[2, ::2] = -INF
    ids, _ = qm.route_scores(logits, k, score=score, normalize=normalize)
    grad = torch.randn(T, k, generator=g, device="cuda")
    if T > 3 and k > 1:
        ids[3, 0] = E + 5       # outside: adds nothing
        ids[0, 1] = ids[0, 0]   # twice the same: both add
    got = qm.route_scores_backward(grad, logits, ids, score=score, normalize=normalize, scale=1.5)
    assert got.dtype == dtype and got.shape == logits.shape
    x, at, d, got = logits.float().cpu().numpy(), ids.cpu().numpy(), grad.cpu().numpy(), got.double().cpu().numpy()
    for t in range(T):
        want, mag = ref.route_grad(x[t], at[t], d[t], score == qm.SCORE_SIGMOID, normalize, 1.5)
        # the weights enter twice; k or E products are added; 1 - s has its own exponential
        tol = (2 * ref.weight_error(x[t], at[t], E) + 2 * k + 16) * ref.U32 * mag
        tol = tol + ref.HALF_STEP[dtype] * (np.abs(want) + tol) + ref.HALF_MIN[dtype] + 2.0 ** -125
        assert np.all(np.abs(got[t] - want) <= tol), (t, np.abs(got[t] - want).max())
        assert np.all(got[t][np.isneginf(x[t])] == 0)


@pytest.mark.parametrize("score", [qm.SCORE_SOFTMAX, qm.SCORE_SIGMOID])
@pytest.mark.parametrize("normalize", [True, False])
def test_gradient_against_differences(score, normalize):
    # the loss's second derivatives are of the order of its first: steps of 2^-6 leave 2^-11 relative, and
    # float32 weights 2^-24 / 2^-6
    T, E, k = 6, 24, 5
    g = torch.Generator(device="cuda").manual_seed(1)
    logits, grad = torch.randn(T, E, generator=g, device="cuda"), torch.randn(T, k, generator=g, device="cuda")
    ids, _ = qm.route_scores(logits, k, score=score, normalize=normalize)
    got = qm.route_scores_backward(grad, logits, ids, score=score, normalize=normalize)
    for t in range(T):
        for e in ids[t, :3].tolist() + [int(logits[t].argmin())]:
            sides = []
            for step in (2.0 ** -6, -2.0 ** -6):
                x = logits.double().cpu().numpy()[t].copy()
                x[e] += step
                w = ref.weights(x, ids[t].cpu().numpy(), score == qm.SCORE_SIGMOID, normalize, 1.0)
                sides.append(float((w * grad[t].double().cpu().numpy()).sum()))
            want = (sides[0] - sides[1]) / 2.0 ** -5
            assert abs(float(got[t, e]) - want) <= 2.0 ** -11 * float(grad[t].abs().sum())


def test_strides_streams_and_graph_replays():
    g = torch.Generator(device="cuda").manual_seed(2)
    wide = torch.randn(300, 100, generator=g, device="cuda").to(BF16)
    x = wide[:, 3:67]
    bias, grad = torch.randn(64, generator=g, device="cuda") * 0.1, torch.randn(300, 4, generator=g, device="cuda")

    def chain(stream=None):
        ids, w = qm.route_scores(x, 4, score=qm.SCORE_SIGMOID, bias=bias, n_groups=8, top_groups=3, group_top=2, stream=stream)
        return ids, w, qm.route_scores_backward(grad, x, ids, score=qm.SCORE_SIGMOID, stream=stream)

    eager = [t.clone() for t in chain()]
    dense = qm.route_scores(x.contiguous(), 4, score=qm.SCORE_SIGMOID, bias=bias, n_groups=8, top_groups=3, group_top=2)
    assert torch.equal(dense[0], eager[0]) and torch.equal(dense[1], eager[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = chain(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, eager))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = chain()
    for _ in range(3):
        wide.copy_(torch.randn(300, 100, generator=g, device="cuda").to(BF16))
        want = [t.clone() for t in chain()]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, want))


def test_no_tokens_and_wrong_tensors():
    x = torch.zeros(0, 8, device="cuda")
    ids, w = qm.route_scores(x, 2)
    assert ids.shape == w.shape == (0, 2)
    assert qm.route_scores_backward(w, x, ids).shape == (0, 8)
    x = torch.zeros(4, 8, device="cuda")
    ids, w = qm.route_scores(x, 2)
    for call in (lambda: qm.route_scores(x.double(), 2), lambda: qm.route_scores(x, 2, bias=x[0, :7]),
                 lambda: qm.route_scores(x, 2, bias=x[0].half()), lambda: qm.route_scores(x[0], 2),
                 lambda: qm.route_scores(x.t(), 2), lambda: qm.route_scores_backward(w, x, ids[:3]),
                 lambda: qm.route_scores_backward(w.half(), x, ids), lambda: qm.route_scores_backward(w[:, :1], x, ids),
                 lambda: qm.route_scores_backward(w, x, ids.long())):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: qm.route_scores(x, 9), lambda: qm.route_scores(x, 2, n_groups=3), lambda: qm.route_scores(x, 0),
                 lambda: qm.route_scores(x, 3, n_groups=4, top_groups=1), lambda: qm.route_scores(x, 2, scale=NAN),
                 lambda: qm.route_scores(x, (1 << 32) + 2)):
        with pytest.raises(qm.QMoEError):
            call()
