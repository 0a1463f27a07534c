"""What the binding of the token operators hands to the library, from tensors of every shape that it takes, and what it refuses.
No GPU needed: the library's call is recorded in place of being made."""
import pytest
import torch

from paged_kv_gqa_block_gb300 import _build


@pytest.fixture
def calls(monkeypatch):
    _build.build()
    import paged_kv_gqa_block_gb300 as pda
    made = []

    def init(self, t, name):
        self.index = t.get_device()      # -1: host memory

    monkeypatch.setattr(pda._Call, "__init__", init)
    monkeypatch.setattr(pda._Call, "run", lambda self, what, fn, p, args, err_word, stream: made.append((what, args)))
    return pda, made


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def pool(p, n=40):
    return torch.zeros(n * p.cache_block_bytes, dtype=torch.uint8)


PATH, WIDTH = 4, 6      # places among accept_tokens' arguments


def test_a_paths_width_is_its_rows(calls):
    """A buffer of more rows than the plan has sequences: the row's length stays the path's."""
    pda, made = calls
    p = pda.plan(4, 2, 8, 16, 8)
    for rows in (4, 8, 11):
        path = i32(rows, 5)
        pda.accept_tokens(p, pool(p), 40, i32(4, 8), i32(4), path, i32(4), i32(4))
        assert made[-1][1][PATH] == path.data_ptr() and made[-1][1][WIDTH] == 5
    empty = pda.plan(0, 2, 8, 16, 8)
    pda.accept_tokens(empty, pool(p), 40, i32(0, 8), i32(0), i32(0, 5), i32(0), i32(0))
    assert made[-1][1][WIDTH] == 5


@pytest.mark.parametrize("shape", [(20,), (3, 5), (2, 2, 5), ()])
def test_paths_of_other_shapes_are_refused(calls, shape):
    pda, made = calls
    p = pda.plan(4, 2, 8, 16, 8)
    with pytest.raises(ValueError, match="path"):
        pda.accept_tokens(p, pool(p), 40, i32(4, 8), i32(4), i32(*shape), i32(4), i32(4))
    assert not made
