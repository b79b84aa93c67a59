"""The give-up paths of the decode over tails and of the fold, each of their waits in turn: in the debug-bounds
build one warp of every CTA is told to give up at a chunk, as if its wait's limit had passed.  The other warps
learn of it through the CTA's flag; copies and MMAs in flight end, tensor memory is freed, the kernel returns and
GLA_ERR_TIMEOUT is reported; the next calls, beside and after it, give what they give without."""
import pytest
import torch

import linear_attention_recurrence_simple_gb300 as gla
from tests.test_gpu_prefix import Case, bits

pytestmark = pytest.mark.gpu
TIMEOUT, UNSUPPORTED, SHAPE = -8, -5, -2


@pytest.fixture(scope="module", autouse=True)
def _setup():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    gla.load_library()
    yield
    assert gla.gla_get_device_error() == 0


@pytest.fixture(scope="module", params=["native", "mxfp8"])
def case(request):
    # tails of no chunk to seventeen (of 32 tokens); the second of four warps has four of the longest's
    lens = [340, 0, 17, 200, 97, 3, 160, 64, 520, 33] * 3
    return Case(970, lens, 4, [i // 4 % 3 for i in range(30)], 3, True, request.param)


def gives_up(call, role, chunk):
    gla.gla_debug_give_up(role, chunk)
    try:
        call()
        return gla.gla_get_device_error()
    finally:
        gla.gla_debug_give_up(-1)


@pytest.mark.parametrize("role, chunk", [(0, 0), (1, 0), (0, 1), (1, 1), (0, 2), (1, 2), (0, 3), (1, 3)])
def test_decode_gives_up(case, role, chunk):
    want = case.decode()
    with gla.debug_bounds_library():
        assert gives_up(case.decode, role, chunk) == TIMEOUT
        assert torch.equal(bits(case.decode()), bits(want))
        assert gives_up(case.decode, role, 4000) == 0    # (no warp has so many chunks)
    assert torch.equal(bits(case.decode()), bits(want))


@pytest.mark.parametrize("role, chunk", [(0, 0), (0, 1), (0, 2), (0, 5), (0, 10), (1, 2), (1, 3), (1, 10), (2, 0), (2, 1), (2, 10)])
def test_fold_gives_up(case, role, chunk):
    want = case.fold()
    with gla.debug_bounds_library():
        assert gives_up(case.fold, role, chunk) == TIMEOUT
        assert torch.equal(case.fold(), want)
    assert torch.equal(case.fold(), want)


def test_a_fold_that_gives_up_leaves_a_decode_on_another_stream_alone(case):
    want_o, want_f = case.decode(), case.fold()
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    with gla.debug_bounds_library():
        gla.gla_debug_give_up(2, 1)
        try:
            case.fold()
            gla.gla_debug_give_up(-1)
            with torch.cuda.stream(other):
                o = case.decode()
        finally:
            gla.gla_debug_give_up(-1)
        torch.cuda.synchronize()
        assert gla.gla_get_device_error() == TIMEOUT
        assert torch.equal(bits(o), bits(want_o)) and torch.equal(case.fold(), want_f)


def test_the_release_build_cannot_be_told_to():
    with pytest.raises(gla.GlaError) as e:
        gla.gla_debug_give_up(0, 0)
    assert e.value.status == UNSUPPORTED
    with gla.debug_bounds_library():
        for role, chunk in ((3, 0), (-2, 0), (0, -1), (0, 4096)):
            with pytest.raises(gla.GlaError) as e:
                gla.gla_debug_give_up(role, chunk)
            assert e.value.status == SHAPE
