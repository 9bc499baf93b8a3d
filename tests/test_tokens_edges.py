"""Edges of the many-token operators' calls that show without a GPU: what an
empty call needs, launches that do not fit, and where the binding allocates."""
import contextlib

import pytest

import sparse_matrix_vector_amd as S

OK, VALUE, OVERFLOW, UNSUPPORTED = 0, 1, 4, 5
P = 4096                                     # a pointer that is aligned and never followed


def test_no_tokens_need_no_workspace():
    L = S.lib()
    for r in (1, 16, 128):
        assert L.lora_apply(0, 64, 32, 3, r, None, None, P, P, 0, None, P, None, 0, None, 64, None, 32, None, 2, 32,
                            None, 0, None) == OK
