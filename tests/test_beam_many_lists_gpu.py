"""Beam selection where many beams over many parts of the vocabulary meet in one merge, and
finished beams whose logits must not be read into the result.  Checked as in test_beam_gpu.py."""
import numpy as np
import pytest
import torch

from test_beam_gpu import DT, check_select

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", [(1, 64, 70001, "f32", 64), (2, 33, 40961, "bf16", 64), (1, 48, 65543, "bf16", 7)],
                         ids=lambda c: "x".join(map(str, c)))
def test_select_over_many_lists(case):
    b, k, V, dtype, count = case
    r = np.random.default_rng(V)
    logits = torch.from_numpy(3 * r.standard_normal((b, k, V))).to(DT[dtype])
    logits[:, 1] = logits[:, 0]  # a row twice: its entries tie where the scores do
    scores = torch.from_numpy(r.uniform(-0.1, 0, (b, k))).float()
    scores[:, 1] = scores[:, 0]
    check_select(logits, scores, count=count)


def test_best_values_side_by_side_in_one_vector():
    """All of a row's best in neighbouring elements, so that one thread holds them all."""
    for V, at in ((9001, 4096), (9001, 8993), (40000, 16383)):
        for dtype in ("bf16", "f32"):
            logits = torch.from_numpy(np.random.default_rng(V).standard_normal((1, 2, V))).to(DT[dtype])
            logits[0, 0, at:at + 8] = torch.arange(8, dtype=torch.float32).to(DT[dtype]) + 20
            check_select(logits, torch.zeros((1, 2)), count=8)


def test_finished_rows_of_nan_do_not_matter():
    r = np.random.default_rng(5)
    logits = torch.from_numpy(r.standard_normal((2, 4, 6000))).to(torch.bfloat16)
    finished = torch.tensor([[True, False, True, False], [True] * 4])
    logits[0, 0] = float("nan")
    logits[1] = float("inf")
    scores = torch.from_numpy(-r.uniform(0, 20, (2, 4))).float()
    check_select(logits, scores, finished=finished, eos=17, count=4)
