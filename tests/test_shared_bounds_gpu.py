"""The decode step over shared prefixes against 64 bits, each term's rounding counted: a bound that a lost step, a wrong mask of the
last step or a missing piece does not pass (tests/test_shared_bounds.py shows that)."""
import numpy as np
import pytest
import torch

from tests import shared_bounds as sb
from tests.shared_cases import CASES, FORMATS, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pda():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_gqa_block_gb300 as pda
    return pda


@pytest.mark.parametrize("kv", FORMATS)
@pytest.mark.parametrize("name", list(CASES))
def test_every_term_is_within_its_rounding(pda, kv, name):
    c = make(name, kv)
    plans = c.plans(pda, **c.plan_kw)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = pda.decode_shared(*plans, **c.device(), out_dtype=torch.float32, err_word=err).double().cpu().numpy()
    assert int(err.item()) == 0
    out, bound = sb.result(c)
    worst = (np.abs(got - out) / bound.clip(1e-300)).max()
    print(f"{name}, format {kv}: {worst:.3f} of the bound")
    assert np.isfinite(got).all() and worst <= 1.0
