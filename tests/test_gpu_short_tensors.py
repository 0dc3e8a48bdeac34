"""GPU: steps over short and misaligned tensors, whose chunks one workgroup takes
alone with the element-wise ends beside the vector part, bit for bit against the
oracle: lengths around every limit (a pack, an element-wise item of 512, a vector
item of 4,096, a chunk), every alignment, both launch forms, the chunk knob."""
import pytest

import adamw_optimizer_step_apply_amd as A
from gpu_util import Case, free, hp_pair

pytestmark = pytest.mark.gpu

SIZES = [1, 6, 7, 8, 9, 15, 16, 17, 255, 256, 257, 511, 512, 513, 519, 2047, 2048, 2056, 4088, 4095, 4096, 4097, 4103,
         4104, 4111, 4112, 6000, 8191, 8192, 8200, 16383, 16384, 16391, 16399, 20_000, 0, 3]
MODES = [("mixed", "bf16"), ("mixed", "f16"), ("kahan", "bf16"), ("split", "bf16"), ("pure-f32-f32-n", "bf16"),
         ("pure-f32-bf16-k", "bf16"), ("pure-bf16-f32-k32", "bf16"), ("pure-bf16-bf16-n", "bf16")]


@pytest.fixture
def knobs():
    yield
    A.adamw_set_single_launch_max_workgroups(-1)
    A.adamw_set_chunk_elems(0)


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
@pytest.mark.parametrize("mode,p_dtype", MODES)
@pytest.mark.parametrize("align", [1, 8])
def test_short_tensors(mode, p_dtype, align, limit, knobs):
    A.adamw_set_single_launch_max_workgroups(limit)
    steps(Case(mode, SIZES, seed=401, p_dtype=p_dtype, align_elems=align, random_moments=True), f"short-{mode}-{align}-{limit}")


@pytest.mark.parametrize("mode,p_dtype", MODES[:4])
@pytest.mark.parametrize("shifts", [{"p": 1, "g": 1, "m": 1, "v": 1}, {"g": 3}, {"p": 8, "g": 16}])
def test_streams_apart(mode, p_dtype, shifts, knobs):
    """Streams that share no 16-byte alignment run element by element."""
    steps(Case(mode, SIZES, seed=402, p_dtype=p_dtype, align_elems=3, random_moments=True, shifts=shifts),
          f"apart-{mode}-{len(shifts)}")


@pytest.mark.parametrize("chunk", [2048, 4096, 1 << 16])
@pytest.mark.parametrize("mode", ["mixed", "kahan", "pure-f32-f32-k"])
def test_chunk_knob(mode, chunk, knobs):
    A.adamw_set_chunk_elems(chunk)
    steps(Case(mode, SIZES + [150_001], seed=403, align_elems=5, random_moments=True), f"knob-{mode}-{chunk}")


@pytest.mark.parametrize("mode", ["mixed", "kahan", "split"])
@pytest.mark.parametrize("shard", [(3, 60_000), (513, 4_700), (16_384, 16_385)])
def test_shard_pieces(mode, shard, knobs):
    case = Case(mode, SIZES, seed=404, align_elems=1, random_moments=True)
    hg, ho = hp_pair()
    case.gpu_step(hg, shard=shard)
    case.oracle_step(ho, shard=shard)
    case.compare_all(f"piece-{mode}-{shard}")
    free()


def test_many_tiny_tensors(knobs):
    """20,000 tensors of 0 to 12 elements: one workgroup each."""
    steps(Case("mixed", [i % 13 for i in range(20_000)], seed=405, align_elems=1, random_moments=True), "tiny", 1)
