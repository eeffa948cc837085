"""Pins of the logits operators' oracle (CPU)."""

import numpy as np
import pytest
import torch

from oracle import logits as ol


def test_adjust_worked_row():
    z = [2.0, -1.0, 0.5, 3.0, 0.0, 1.0]
    got = ol.adjust_row(z, counts={0: 2, 3: 1}, prompt=[1, 3], drafts=[3, 5], repetition=2.0, presence=0.25,
                        frequency=0.5, bias=[(2, 1.5), (2, -1.0), (9, 7.0)], allowed=[1, 1, 1, 1, 0, 1])
    # 0: 2/2 - 0.5*2 - 0.25; 1: prompt only, -1*2; 2: two biases; 3: 3/2 - 0.5*2 - 0.25; 4 masked; 5: a draft
    assert got.tolist() == [-0.25, -2.0, 1.0, 0.25, -np.inf, -0.25]


def test_adjust_masks_everything_and_nan():
    got = ol.adjust_row([np.nan, np.inf, 1.0], allowed=[False, False, False])
    assert (got == -np.inf).all()


def test_top_logits_order_and_sums():
    z = np.array([1.0, 5.0, 5.0, -np.inf, 2.0, 5.0])
    tok, val, lse, rest = ol.top_logits(z, 2, 0.5)
    assert tok.tolist() == [1, 2] and val.tolist() == [5.0, 5.0]
    assert lse == pytest.approx(np.log(np.exp(2 * z).sum()), rel=1e-15)
    assert rest == pytest.approx(np.log(np.exp(2 * z[[0, 4, 5]]).sum()), rel=1e-15)
    tok, val, lse, rest = ol.top_logits(z[:2], 4, 1.0)
    assert tok.tolist() == [1, 0, -1, -1] and rest == -np.inf
    assert np.isnan(ol.top_logits([np.nan, 1.0], 1, 1.0)[2])


def _case(seed, V=40, K=6, T=1.7):
    rng = np.random.default_rng(seed)
    teacher, student = rng.normal(0, 3, V), rng.normal(0, 3, V)
    return student, *ol.top_logits(teacher, K, T), T


@pytest.mark.parametrize("tail", ["bucket", "renorm"])
@pytest.mark.parametrize("duplicate", [False, True])
def test_gradient_against_differences(tail, duplicate):
    z, tok, val, lse, rest, T = _case(3)
    if duplicate:
        tok, val = np.append(tok, [tok[1], -1, 40]), np.append(val, [val[1] - 1, 2.0, 2.0])
    loss, grad, _, ok = ol.distill(z, tok, val, (lse, rest), T, tail, w=0.3)
    assert ok
    h = 1e-5
    for v in range(len(z)):
        d = np.zeros(len(z))
        d[v] = h
        num = (ol.distill(z + d, tok, val, (lse, rest), T, tail, 0.3)[0]
               - ol.distill(z - d, tok, val, (lse, rest), T, tail, 0.3)[0]) / (2 * h)
        # central difference: error h^2 / 6 of a third derivative below 1, and 2 ulp of the loss over 2 h
        assert abs(num - grad[v]) < 1e-9, v


@pytest.mark.parametrize("tail", ["bucket", "renorm"])
def test_whole_vocabulary_record_is_the_kl_divergence(tail):
    rng = np.random.default_rng(5)
    V, T = 30, 0.8
    t, z = rng.normal(0, 2, V), rng.normal(0, 2, V)
    tok, val, lse, rest = ol.top_logits(t, V, T)
    assert rest == -np.inf
    loss, grad, _, _ = ol.distill(z, tok, val, (lse, rest), T, tail)
    x = torch.tensor(z, dtype=torch.float64, requires_grad=True)
    kl = torch.nn.functional.kl_div(torch.log_softmax(x / T, 0), torch.softmax(torch.tensor(t) / T, 0),
                                    reduction="sum")
    kl.backward()
    assert loss == pytest.approx(kl.item(), rel=1e-12)
    assert np.allclose(grad, x.grad.numpy(), rtol=1e-10, atol=1e-14)


def test_student_equal_to_the_teacher_has_no_loss():
    rng = np.random.default_rng(6)
    t = rng.normal(0, 3, 100)
    tok, val, lse, rest = ol.top_logits(t, 10, 1.0)
    loss, grad, _, _ = ol.distill(t, tok, val, (lse, rest), 1.0, "bucket")
    assert abs(loss) < 1e-14 and np.abs(grad).max() < 1e-15


def test_planted_mistakes_are_seen():
    # the rest's term left out of the gradient, and the temperature left out: the difference test must see both
    z, tok, val, lse, rest, T = _case(4)
    _, grad, _, _ = ol.distill(z, tok, val, (lse, rest), T, "bucket")
    wrong = ol.distill(z, tok, val, (lse, -np.inf), T, "bucket")[1]
    assert np.abs(wrong - grad).max() > 1e-3
    assert np.abs(grad * T - grad).max() > 1e-3


def test_left_out_rows():
    z = np.array([0.5, 1.0, 2.0])
    for tok, val, lse in (([-1, 7], [1.0, 1.0], (0.0, 0.0)), ([0, 1], [np.nan, 1.0], (0.0, 0.0)),
                          ([0, 1], [-np.inf, -np.inf], (0.0, 0.0))):
        loss, grad, _, ok = ol.distill(z, tok, val, lse, 1.0, "renorm")
        assert loss == 0 and not grad.any() and not ok
    loss, grad, _, ok = ol.distill(z, [0], [1.0], (np.nan, np.nan), 1.0, "bucket")
    assert loss == 0 and not grad.any() and not ok
    loss, grad, _, ok = ol.distill([np.nan, 1.0], [0], [1.0], (1.5, 0.0), 1.0, "bucket")
    assert np.isnan(loss) and np.isnan(grad).all() and not ok
