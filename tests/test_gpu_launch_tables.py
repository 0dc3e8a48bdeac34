"""GPU: steps over lists on both sides of the limit at which a short chunk becomes one
workgroup's, bit for bit against the oracle: lists that fit on the card whole (every chunk
shared, the ends of a tensor by themselves) and lists that do not (short chunks alone, the
ends with their vector chunks), in every kernel family and both launch forms."""
import pytest

import adamw_optimizer_step_apply_amd as A
from gpu_util import Case, free, hp_pair
from test_gpu_short_tensors import MODES, SIZES, knobs  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu

ALL = MODES + [("pure-bf16-f32-n", "bf16"), ("pure-f32-f32-k32", "bf16"), ("pure-bf16-bf16-k", "bf16")]


def steps(case, label, n=2):
    hg, ho = hp_pair()
    for s in range(n):
        if s:
            case.refill_grads(s)
        case.gpu_step(hg)
        case.oracle_step(ho)
    case.compare_all(label)
    free()


@pytest.mark.parametrize("limit", [-1, 0])
@pytest.mark.parametrize("mode,p_dtype", ALL)
@pytest.mark.parametrize("align", [1, 8])
def test_many_short_tensors(mode, p_dtype, align, limit, knobs):  # noqa: F811
    A.adamw_set_single_launch_max_workgroups(limit)
    case = Case(mode, SIZES * 6, seed=431, p_dtype=p_dtype, align_elems=align, random_moments=True)
    assert 8 * sum(n > 0 for n in case.numels) > 1024     # workgroups, 8 a chunk: more than the card holds at once
    steps(case, f"many-{mode}-{align}-{limit}")


@pytest.mark.parametrize("limit", [-1, 0])
@pytest.mark.parametrize("mode,p_dtype", ALL)
@pytest.mark.parametrize("align", [1, 8])
def test_few_short_tensors(mode, p_dtype, align, limit, knobs):  # noqa: F811
    A.adamw_set_single_launch_max_workgroups(limit)
    for k, n in enumerate((1, 7, 9, 12, 100, 128, 135, 700, 2055, 4096, 4110, 8200)):
        steps(Case(mode, [n, 3, n], seed=432 + k, p_dtype=p_dtype, align_elems=align, random_moments=True),
              f"few-{mode}-{align}-{limit}-{n}", 1)


@pytest.mark.parametrize("chunks", [63, 64, 65, 127, 128, 129])
@pytest.mark.parametrize("mode", ["mixed", "kahan", "split", "pure-f32-f32-k32"])
def test_around_the_limit(mode, chunks, knobs):  # noqa: F811
    """One vector chunk per tensor, and one more list entry than the limit."""
    steps(Case(mode, [1024 + 8 * (i % 5) for i in range(chunks)], seed=433, align_elems=8, random_moments=True),
          f"limit-{mode}-{chunks}", 1)
