"""int8 experts' workspace as include/dwdp.h lays it out: A's codes, scales and fp32 values, then the schedule."""
import numpy as np
import pytest
import torch


def align(n):
    return (n + 255) // 256 * 256


def places(rows, I):
    """Offsets of A's scales and fp32 values, and of what follows them."""
    scale = align(rows * I)
    values = scale + align(rows * 4)
    return scale, values, values + align(rows * I * 4)


@pytest.mark.parametrize("rows,I", [(1, 128), (63, 128), (64, 256), (1000, 768), (73728, 2048)])
def test_size(rows, I):
    from split_weight_expert_amd import api

    def size(dtype):
        return api.workspace_bytes(api.OP_GROUPED_FFN, rows, 1, 5, 256, I, dtype, 0)
    # bf16 has A alone before the same schedule
    assert size(api.INT8) - places(rows, I)[2] == size(api.BF16) - align(rows * I * 2)
    if rows > 1000:
        assert 2.45 < size(api.INT8) / size(api.BF16) < 2.51


@pytest.mark.gpu
@pytest.mark.parametrize("rows,H,I", [([5], 256, 128), ([33, 0, 64, 7], 512, 384), ([300, 129], 256, 1152)])
def test_codes_are_those_of_the_fp32_values(rows, H, I):
    """A's codes and scales are, bit for bit, the quantiser's of the fp32 A beside them."""
    from oracle import int8 as o8
    from split_weight_expert_amd import api
    from tests.test_gpu_int8 import Layer, U
    L = Layer(api, rows, H, I, 3)
    L.run(1)
    scale, values, end = places(L.n, I)
    assert end <= L.ws.numel()
    a32 = L.ws[values:values + 4 * L.n * I].view(torch.float32).view(L.n, I).cpu().numpy()
    codes, scales = o8.rows(a32)
    np.testing.assert_array_equal(L.ws[:L.n * I].view(torch.int8).view(L.n, I).cpu().numpy(), codes)
    np.testing.assert_array_equal(L.ws[scale:scale + 4 * L.n].view(torch.float32).cpu().numpy(), scales)
    for e in range(L.G):
        r = slice(int(L.off[e]), int(L.off[e + 1]))
        src = L.src[r].numpy()
        A, gate = o8.gate_up(L.q.cpu().numpy()[src], L.qs.cpu().numpy()[src], L.w13[e].numpy(), L.s13[e].numpy())
        assert (np.abs(a32[r] - A) <= np.abs(A) * (3.5 * np.abs(gate) + 12) * 2 * U).all()
