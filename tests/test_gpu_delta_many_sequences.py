"""Packed bf16 calls of the gated delta rule around the number of sequences up to which they are put in order: every
sequence's results are those of a call of its own kind with the sequences in groups."""
import pytest
import torch

import linear_attention_recurrence_simple_gb300 as gla
from tests.delta_helpers import DK, DV

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _setup():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    gla.load_library()
    yield
    assert gla.gla_get_device_error() == 0


def inputs(lens, H):
    g = torch.Generator(device="cuda").manual_seed(51)
    T = int(lens.sum())
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    unit = torch.nn.functional.normalize
    return [unit(r(T, H, DK), dim=-1).to(BF), unit(r(T, H, DK), dim=-1).to(BF), r(T, H, DV).to(BF), -r(T, H).abs().to(BF),
            torch.sigmoid(r(T, H)).to(BF)], r(T, H, DV).to(BF)


def offsets(lens):
    return torch.cat([lens.new_zeros(1), lens.cumsum(0)]).to(torch.int32).cuda()


@pytest.mark.parametrize("N", [16384, 16385])
def test_as_in_groups(N):
    lens = torch.randint(0, 4, (N,), generator=torch.Generator().manual_seed(52))
    lens[[5, 9000, N - 1]] = torch.tensor([130, 64, 200])
    H = 1
    x, dO = inputs(lens, H)
    h0 = (torch.randn(N, H, DK, DV, generator=torch.Generator(device="cuda").manual_seed(53), device="cuda") * 0.1)
    o, hT = gla.gla_delta_fwd(*x, h0=h0, cu_seqlens=offsets(lens))
    grads = gla.gla_delta_bwd(*x, dO, h0=h0, cu_seqlens=offsets(lens))
    ends = lens.cumsum(0)
    for lo in range(0, N, 5000):
        hi = min(N, lo + 5000)
        t = slice(int(ends[lo] - lens[lo]), int(ends[hi - 1]))
        cu, part = offsets(lens[lo:hi]), [y[t] for y in x]
        o2, hT2 = gla.gla_delta_fwd(*part, h0=h0[lo:hi], cu_seqlens=cu)
        assert torch.equal(o[t], o2) and torch.equal(hT[lo:hi], hT2)
        grads2 = gla.gla_delta_bwd(*part, dO[t], h0=h0[lo:hi], cu_seqlens=cu)
        for a, c in zip(grads[:5], grads2):
            assert torch.equal(a[t], c)
        assert torch.equal(grads[5][lo:hi], grads2[5])


def test_time_grows_with_the_sequences():
    """Four times the sequences take at most six times as long (four and what varies; compared pair by pair, half a million
    took nine times what 131,072 did)."""
    def us(N):
        x, _ = inputs(torch.ones(N, dtype=torch.int64), 1)
        cu = offsets(torch.ones(N, dtype=torch.int64))
        ws = torch.empty(gla.gla_delta_workspace_bytes(N, N, 1, True, 0), dtype=torch.uint8, device="cuda")
        times = []
        for _ in range(4):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            gla.gla_delta_fwd(*x, cu_seqlens=cu, output_final_state=False, workspace=ws)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)

    small, large = us(1 << 17), us(1 << 19)
    print(f"{small:.2f} ms, {large:.2f} ms")
    assert large <= 6 * small
