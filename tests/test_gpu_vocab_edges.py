"""The loss over a vocabulary at the edges of its layouts and values. Bounds as in
test_gpu_vocab.py, unless a test derives its own."""
import math

import pytest
import torch

from gpu_util import say
from test_gpu_vocab import check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,stride", [(25, 26), (1, 2), (63, 70)], ids=str)
def test_rows_of_odd_length_at_even_strides(dim, stride):
    """bf16 rows that end between words, the last one at the end of its memory."""
    say("case vocab odd rows %d %d" % (dim, stride))
    x, W, target, dloss = make(dim, "bf16", 133, dim, 300, False)
    memory = torch.full((132 * stride + dim,), float("nan"), dtype=torch.bfloat16, device="cuda")
    rows = memory.as_strided((133, dim), (stride, 1))
    rows.copy_(x)
    check(rows, W, target, dloss)
