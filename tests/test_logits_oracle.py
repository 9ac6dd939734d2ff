"""Pins of the host definitions of the operators on rows of logits (no GPU)."""
import math

import numpy as np
import pytest

from oracle import logits_ref as ref


def test_top_logits_by_hand():
    ids, lp, lse = ref.top_logits([1.0, 3.0, -np.inf, 3.0], 5)
    assert list(ids) == [1, 3, 0, -1, -1]
    assert lse == pytest.approx(math.log(math.e + 2 * math.e ** 3), abs=1e-14)
    assert lp[2] == pytest.approx(1.0 - lse, abs=1e-14) and lp[3] == -np.inf
    ids, _, lse = ref.top_logits([1.0, 3.0, 2.0], 2, mask=np.array([True, False, True]))
    assert list(ids) == [2, 0] and lse == pytest.approx(math.log(math.e + math.e ** 2), abs=1e-14)
    ids, _, lse = ref.top_logits([np.nan, 5.0], 2)
    assert list(ids) == [1, -1] and np.isnan(lse)


def test_a_label_is_the_cross_entropy():
    z = np.random.default_rng(0).standard_normal(50)
    for rest in (False, True):
        loss, (every, _), grad, _ = ref.distill(z, [7], [0.0], rest=rest)
        assert loss == pytest.approx(every - z[7], rel=1e-13)
        want = np.exp(z - every)
        want[7] -= 1
        assert np.allclose(grad, want, atol=1e-14)


def test_a_drafter_like_its_target_has_no_loss():
    z = np.random.default_rng(1).standard_normal(60) * 3
    ids, lp, _ = ref.top_logits(z, 9, temperature=1.5)
    loss, _, grad, ratio = ref.distill(z, ids, lp, temperature=1.5)
    assert abs(loss) < 1e-14 and np.abs(grad).max() < 1e-14 and ratio == pytest.approx(1.0, rel=1e-12)


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("tau", [0.7, 1.0, 2.5])
def test_distillation_gradient_against_differences(rest, tau):
    """A central difference of step h is off by h^2 / 6 times a third derivative (under 16 / tau^3) and by the loss's own
    rounding, 2^-50 or so, over h."""
    rng = np.random.default_rng(2)
    z = rng.standard_normal(40) * 2
    ids, lp, _ = ref.top_logits(z + rng.standard_normal(40), 6, temperature=tau)
    _, _, grad, _ = ref.distill(z, ids, lp, tau, rest, 0.3)
    h = 1e-4
    for j in list(ids[:3]) + [int(x) for x in np.setdiff1d(np.arange(40), ids)[:5]]:
        up, down = z.copy(), z.copy()
        up[j] += h
        down[j] -= h
        d = (ref.distill(up, ids, lp, tau, rest, 0.3)[0] - ref.distill(down, ids, lp, tau, rest, 0.3)[0]) / (2 * h)
        assert abs(d - grad[j]) <= h * h * 16 / tau ** 3 + 2.0 ** -46 / h


def test_entries_that_do_not_count():
    ids, lps, fault = ref.entries([3, -1, 3, 50, 4, 5], [-1.0, np.nan, -2.0, -1.0, np.nan, -np.inf], 50)
    assert list(ids) == [3, 5] and list(lps) == [-1.0, -np.inf] and fault
    assert not ref.entries([3, -1], [-1.0, np.nan], 50)[2]


def test_beams_against_the_whole_list():
    rng = np.random.default_rng(3)
    z, scores = rng.standard_normal((3, 20)), np.array([-1.0, -np.inf, -1.5])
    beams, tokens, got, ended, _ = ref.beam_select(z, scores, 4, end_token=5)
    full = scores[:, None] + z - np.array([ref.log_sum(r) for r in z])[:, None]
    order = np.argsort(-full, axis=None, kind="stable")[:4]
    assert beams == list(order // 20) and tokens == list(order % 20) and np.allclose(got, full.reshape(-1)[order])
    assert ended == [int(t == 5) for t in tokens]
    beams, tokens, got, ended, _ = ref.beam_select(z[:1], [-2.0], 3, finished=[1], end_token=5)
    assert (beams, tokens, got, ended) == ([0, -1, -1], [5, -1, -1], [-2.0, -np.inf, -np.inf], [1, 0, 0])
