"""Which padding ids the embedding takes (CPU only: the refusal comes before the tensors are looked at)."""
from __future__ import annotations

import pytest
import torch

import linear_cross_entropy_tmem_gb300 as F


@pytest.mark.parametrize("padding", [-1, -2, -4, -(1 << 40)])
def test_negative_padding_ids_are_refused(padding):
    """torch.nn.functional.embedding counts them from the table's end; taken as "none" they would lose the padding row's
    exclusion without a word."""
    w, ids = torch.zeros(4, 64), torch.zeros(2, dtype=torch.int64)
    for call in (lambda: F.embedding(w, ids, padding_idx=padding), lambda: F.Embedding.apply(w, ids, 1.0, padding, None),
                 lambda: F.flce_embedding_backward(w[:2], ids, 4, padding_idx=padding)):
        with pytest.raises(ValueError, match="padding_idx.*not counted from its end"):
            call()


@pytest.mark.parametrize("padding", [None, 0, 3, 4])
def test_others_come_to_the_tensors(padding):
    w, ids = torch.zeros(4, 64), torch.zeros(2, dtype=torch.int64)
    for call in (lambda: F.embedding(w, ids, padding_idx=padding),
                 lambda: F.flce_embedding_backward(w[:2], ids, 4, padding_idx=padding)):
        with pytest.raises(RuntimeError, match="CUDA"):
            call()
