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


def half(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


@pytest.mark.parametrize("shape,tokens", [((7, 2, 128), 7), ((0, 2, 128), 0), ((7, 256), 7), ((7 * 256,), 7), ((1, 7, 2, 128), 7)])
def test_read_kv_takes_whole_tokens(calls, shape, tokens):
    pda, made = calls
    p = pda.plan(3, 2, 8, 16, 8)
    for outs in ((half(*shape), half(*shape)), (half(*shape), None), (None, half(*shape))):
        pda.read_kv(p, pool(p), 40, i32(3, 8), i32(4), i32(3), *outs)
        assert made[-1][1][6] == tokens


@pytest.mark.parametrize("shape", [(7, 2, 127), (1000,), (7, 4, 128), (14, 1, 128), (7, 128, 2, 3)])
def test_read_kv_refuses_parts_of_tokens_and_other_heads(calls, shape):
    """Not the whole tokens in front of a remainder, and not 14 tokens of one head as 7 of two."""
    pda, made = calls
    p = pda.plan(3, 2, 8, 16, 8)
    for outs in ((half(*shape), None), (None, half(*shape))):
        with pytest.raises(ValueError, match="tokens"):
            pda.read_kv(p, pool(p), 40, i32(3, 8), i32(4), i32(3), *outs)
    assert not made


@pytest.mark.parametrize("shape,tokens", [((5, 16, 128), 5), ((5, 2, 8, 128), 5), ((0, 16, 128), 0), ((5 * 2048,), 5)])
def test_decode_tree_takes_whole_tokens(calls, shape, tokens):
    pda, made = calls
    p = pda.plan(3, 2, 8, 16, 8)
    pda.decode_tree(p, half(*shape), pool(p), 40, i32(3, 8), i32(3), i32(4))
    assert made[-1][1][1] == tokens and made[-1][1][13] == pda.lib().pda_tree_workspace_size(p, tokens)


@pytest.mark.parametrize("shape", [(5, 16, 127), (5000,), (5, 32, 128), (10, 8, 128)])
def test_decode_tree_refuses_other_queries(calls, shape):
    pda, made = calls
    p = pda.plan(3, 2, 8, 16, 8)
    with pytest.raises(ValueError, match="query"):
        pda.decode_tree(p, half(*shape), pool(p), 40, i32(3, 8), i32(3), i32(4))
    assert not made


@pytest.mark.parametrize("name", ["window", "num_first"])
@pytest.mark.parametrize("value", [1 << 31, (1 << 32) + 16, 1 << 63, -(1 << 31) - 1, -(1 << 32) + 16])
def test_windows_past_32_bits_are_refused(calls, name, value):
    """Not taken modulo 2^32, as a window of 16."""
    pda, made = calls
    p = pda.plan(3, 2, 8, 16, 8)
    kw = dict(window=100, num_first=4)
    kw[name] = value
    with pytest.raises(ValueError, match=name):
        pda.decode_tree(p, half(5, 16, 128), pool(p), 40, i32(3, 8), i32(3), i32(4), **kw)
    with pytest.raises(ValueError, match=name):
        pda.decode_window(p, half(3, 16, 128), pool(p), 40, i32(3, 8), i32(3), **kw)
    assert not made
    pda.decode_tree(p, half(5, 16, 128), pool(p), 40, i32(3, 8), i32(3), i32(4), window=(1 << 31) - 1, num_first=(1 << 31) - 1)
    assert made[-1][1][10:12] == ((1 << 31) - 1, (1 << 31) - 1)
