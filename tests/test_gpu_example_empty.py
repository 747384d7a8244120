"""The example's scoring of no rows: every result with its columns, and no rows."""
import pytest
import torch

import invariant_token_log_gb300 as bil
from test_gpu_example import data, example  # noqa: F401

pytestmark = pytest.mark.gpu


def test_score_of_no_rows(example):  # noqa: F811
    x, r, w, weight, t = data(3, 128, 1000)
    wq, ws = bil.quantize_rows(weight)
    want = example.score(x, r, w, wq, ws, t, k=7)
    got = example.score(x[:0], r[:0], w, wq, ws, t[:0], k=7)
    for a, b in zip(got, want):
        assert a.shape == (0, *b.shape[1:]) and a.dtype == b.dtype
