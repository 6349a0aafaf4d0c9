"""What a block keeps between its calls, without a GPU: the library's calls are replaced by recorders."""
import pytest
import torch

from split_weight_expert_amd import MoEBlock, api


class Calls(list):
    """Names of the library calls made; a name in `refuse` raises as a refused call does."""
    refuse = ()


@pytest.fixture
def calls(monkeypatch):
    seen = Calls()

    def stub(name):
        def f(*a, **kw):
            if name in seen.refuse:
                raise ValueError(f"{name} refused")
            seen.append(name)
        return f
    for name in ("route_gate", "route_topk", "permute", "quantize_tokens_fp8", "moe_grouped_ffn_stage", "moe_grouped_ffn_tokens",
                 "combine", "add_rmsnorm", "combine_add_rmsnorm"):
        monkeypatch.setattr(api, name, stub(name))
    return seen


def block(dtype="bf16", **kw):
    return MoEBlock(256, 128, 8, 2, 0, dtype, "cpu", **kw)


def rows(T=4):
    return torch.zeros(T, 256, dtype=torch.bfloat16)


def test_methods_have_their_docstrings():
    for name in ("forward", "permute", "norm", "forward_normed"):
        assert getattr(MoEBlock, name).__doc__, name


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8"])
def test_a_norm_refused_after_another_is_none(calls, dtype):
    blk = block(dtype)
    x, w, b = rows(), torch.ones(256), blk.buffers(4)
    blk.norm(x, w, 1e-6, b)
    blk.forward_normed(x, None, None, None)
    blk.norm(x, w, 1e-6, b)
    calls.refuse = ("add_rmsnorm",)
    with pytest.raises(ValueError, match="add_rmsnorm refused"):
        blk.norm(x, w, 1e-6, b)
    with pytest.raises(ValueError, match="no normed input"):
        blk.forward_normed(x, None, None, None)
