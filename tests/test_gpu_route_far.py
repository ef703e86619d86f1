"""GPU tests of the choice of experts where scores in 64 bits round to the same number: without a bias experts are compared by
their logits, groups by their scores."""
import pytest
import torch

import i8_reference as ref
import tiled_dense_gemm_fp16_amd as g

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def chosen(rows, top_k, score, bias=None, **kw):
    x = torch.tensor(rows)
    b = None if bias is None else torch.tensor(bias, device=DEV)
    ids, weights = g.route(x.to(DEV), top_k, score=score, bias=b, **kw)
    want_ids, want = ref.route(x.numpy(), top_k, score, bias, **kw)
    assert (ref.host(ids) == want_ids).all() and (abs(ref.host(weights) - want) <= want * 2.0 ** -22).all()
    return ref.host(ids).tolist()


def test_equal_scores():
    rows = [[40.0, 60.0, 50.0, 45.0]]                      # sigmoids of 1 in 64 bits
    assert chosen(rows, 3, "sigmoid") == [[1, 2, 3]]       # by logit
    assert chosen(rows, 3, "sigmoid", [0.0] * 4) == [[0, 1, 2]]   # by score + bias
    rows = [[0.0, -900.0, -800.0, -850.0]]                 # softmaxes of 0 behind the first
    assert chosen(rows, 3, "softmax") == [[0, 2, 3]]
    assert chosen(rows, 3, "softmax", [0.0] * 4) == [[0, 1, 2]]


@pytest.mark.parametrize("score,row", [("sigmoid", [40.0, 41.0, 60.0, 70.0, 50.0, 51.0]),
                                       ("softmax", [-900.0, -890.0, -800.0, -790.0, 0.0, -1e4])])
def test_groups_of_equal_scores(score, row):
    """Of groups whose scores have the same sum the first stay, whatever their logits; inside them logits decide."""
    first = [4, 5] if score == "softmax" else [1, 0]
    assert chosen([row], 2, score, groups=3, top_groups=1) == [first]
    both = [4, 1, 0] if score == "softmax" else [3, 2, 1]
    assert chosen([row], 3, score, groups=3, top_groups=2) == [both]
