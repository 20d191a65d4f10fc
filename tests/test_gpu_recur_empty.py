"""The recurrence over packed sequences most of which are empty, in long runs that
fall inside blocks of 16 rows, on their borders and at either end: the others'
results, and the states passed through."""
import pytest
import torch

import ternary_weight_linear_tern_amd as tl
from gpu_util import log
from test_gpu_recur import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    tl.lib()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("act,dy", [("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("lens", [[100] + [0] * 40000 + [60, 1] + [0] * 1000 + [3, 300],
                                  [0] * 5000 + [128] + [0] * 63 + [16] + [0] * 65 + [700] + [0] * 5000])
def test_long_runs_of_empty_sequences(lens, act, dy):
    log(f"recur {len(lens)} sequences, {act}")
    c = Case(sum(lens) + 5, 40, act, lens, False, dy, seed=len(lens))
    c.fwd()
    c.bwd()
    c.check()
