"""What a block keeps between its calls, without a GPU: the library's calls are replaced by recorders."""
import pytest
import torch

pytest.importorskip("split_weight_expert_amd._lib")

from split_weight_expert_amd import MoEBlock, api  # noqa: E402


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


def forward(blk, h, **kw):
    return blk.forward_normed(h, None, None, None, **kw)


def refused(calls, blk, h, **kw):
    n = len(calls)
    with pytest.raises(ValueError, match="no normed input"):
        forward(blk, h, **kw)
    assert len(calls) == n, "a refused call made others"


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8"])
@pytest.mark.parametrize("gather", [False, True])
def test_two_batches_of_one_size(calls, dtype, gather):
    """The second norm took the first one's place: only the second batch's layer runs."""
    blk = block(dtype, gather=gather)
    h1, h2, w, b = rows(), rows(), torch.ones(256), blk.buffers(4)
    n1 = blk.norm(h1, w, 1e-6, b)
    n2 = blk.norm(h2, w, 1e-6, b)
    refused(calls, blk, h1)
    refused(calls, blk, h1, normed=n1)
    refused(calls, blk, h2.clone())
    forward(blk, h2)
    forward(blk, h2.view(4, 256))             # another view of the same rows
    forward(blk, h2, normed=n2)
    forward(blk, h1, normed=n2)               # with the handle the caller says whose norm it is
    assert calls.count("combine_add_rmsnorm") == 4
    # a batch of another size has its own
    h3 = rows(6)
    refused(calls, blk, h3)
    blk.norm(h3, w, 1e-6, blk.buffers(6))
    forward(blk, h3)
    forward(blk, h2)


def test_layers_hand_their_norm_on(calls):
    blk = block()
    x, w, b = rows(), torch.ones(256), blk.buffers(4)
    o1, o2 = rows(), rows()
    n = blk.norm(x, w, 1e-6, b)
    assert forward(blk, x, next_weight=w, out=o1).normed is not n
    refused(calls, blk, x)                    # the buffers hold o1's norm now
    refused(calls, blk, x, normed=n)
    forward(blk, o1, next_weight=w)           # to b.y
    refused(calls, blk, o1)
    forward(blk, b.y, out=o2)                 # the last layer
    refused(calls, blk, x)                    # the next request was not normed
    refused(calls, blk, o2)
    forward(blk, b.y, out=o2)                 # the same one's input is still there


def test_writes_to_the_normed_tensor(calls):
    blk = block()
    x, w, b = rows(), torch.ones(256), blk.buffers(4)
    blk.norm(x, w, 1e-6, b)
    forward(blk, x)
    x.copy_(torch.ones(4, 256))               # the next request in the same memory
    refused(calls, blk, x)
    n = blk.norm(x, w, 1e-6, b)
    x.add_(1)                                 # a parallel branch's sum: x is not what was normed, the handle says it is meant
    refused(calls, blk, x)
    forward(blk, x, normed=n)
    blk.norm(x, w, 1e-6, b)
    forward(blk, x, out=x)                    # in place: the layer wrote it
    refused(calls, blk, x)
    n = blk.norm(x, w, 1e-6, b)
    forward(blk, rows(), normed=n, out=x)
    refused(calls, blk, x)
    blk.norm(x, w, 1e-6, b)
    forward(blk, x, next_weight=w, out=x)     # in place, with the next norm
    forward(blk, x, out=x)
    refused(calls, blk, x)
    blk.norm(x, w, 1e-6, b)
    forward(blk, x, out=b.x_norm)             # the normed input itself was overwritten
    refused(calls, blk, x)


def test_freed_memory_is_no_batch(calls):
    blk = block()
    w, b = torch.ones(256), blk.buffers(4)
    x = rows()
    at = x.data_ptr()
    blk.norm(x, w, 1e-6, b)
    del x
    for _ in range(50):                       # some allocation usually gets the same address
        y = rows()
        refused(calls, blk, y)
        if y.data_ptr() == at:
            break


def test_sums_and_their_handles(calls):
    blk = block()
    x, r, s, w, b = rows(), rows(), rows(), torch.ones(256), blk.buffers(4)
    blk.norm(x, w, 1e-6, b, residual=r, sum_out=s)
    forward(blk, s)
    refused(calls, blk, x)
    refused(calls, blk, r)
    n = blk.norm(x, w, 1e-6, b, residual=r, sum_out=r)        # in place
    forward(blk, r)
    n = blk.norm(x, w, 1e-6, b, residual=r)                   # the sum is nobody's: by its handle alone
    refused(calls, blk, x)
    refused(calls, blk, x + r)
    forward(blk, x + r, normed=n)
    blk.forward(x, None, None, None)
    refused(calls, blk, x + r, normed=n)


def test_inference_tensors(calls):
    blk = block()
    w, b = torch.ones(256), blk.buffers(4)
    with torch.inference_mode():
        x = rows()
        blk.norm(x, w, 1e-6, b)
        forward(blk, x)
        refused(calls, blk, rows())


def test_a_refused_boundary_leaves_no_normed_input(calls):
    """A layer that failed at its end may have left anything in the buffers; one refused before has touched nothing."""
    blk = block()
    x, w, b = rows(), torch.ones(256), blk.buffers(4)
    blk.norm(x, w, 1e-6, b)
    calls.refuse = ("route_topk",)
    with pytest.raises(ValueError, match="route_topk refused"):
        forward(blk, x)
    calls.refuse = ("combine_add_rmsnorm",)
    with pytest.raises(ValueError, match="combine_add_rmsnorm refused"):
        forward(blk, x)
    calls.refuse = ()
    refused(calls, blk, x)


def test_copies_of_a_block(calls):
    """A copied or stored normed input knows no tensor: its own handle is needed, and nothing is freed twice."""
    import copy
    import io
    import pickle
    blk = block()
    x, w, b = rows(), torch.ones(256), blk.buffers(4)
    n = blk.norm(x, w, 1e-6, b)
    f = io.BytesIO()
    pickle.dump(n, f)
    assert n._memory is not None and pickle.loads(f.getvalue())._memory is None and copy.copy(n)._memory is None
    other = copy.deepcopy(blk)
    o = other.buffers(4).normed
    assert o is not n and o._memory is None
    refused(calls, other, x)
    refused(calls, other, x, normed=n)
    forward(other, x, normed=o)
    del other, o
    forward(blk, x)
