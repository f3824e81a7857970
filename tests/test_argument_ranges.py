"""Numbers that do not fit the C interface's types are refused or counted as what
they mean, never cut to their lower bits."""
import ctypes

import pytest
import torch

from encoder_only_transformer_gb300 import binding


@pytest.fixture(scope="module")
def built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("dim", [2 ** 32 + 64, -2 ** 32 + 64, 2 ** 31, 2 ** 63 + 2])
def test_rotary_dim_beyond_32_bits(built, dim):
    with pytest.raises(binding.MbertAttnError):
        binding.Rotary(dim)


def test_rotary_dim_is_whole(built):
    with pytest.raises(ValueError):
        binding.Rotary(64.9)
    assert binding.Rotary(64.0).dim == 64 and binding.Rotary(torch.tensor(64)).dim == 64


@pytest.mark.gpu
@pytest.mark.parametrize("bound", [2 ** 32 + 1, 2 ** 31, 2 ** 63])
def test_query_bound_beyond_32_bits(built, bound):
    """A bound larger than any sequence is no bound: not its lower bits (1)."""
    q = torch.randn(3, 2, 64, device="cuda").bfloat16()
    kv = torch.randn(10, 2, 64, device="cuda").bfloat16()
    cq = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    ck = torch.tensor([0, 10], dtype=torch.int32, device="cuda")
    want = binding.cross_attention(q, kv, kv, cq, ck)
    got = binding.cross_attention(q, kv, kv, cq, ck, max_seqlen_q=bound)
    assert binding._default(q.device).get_error() == 0 and torch.equal(got, want)
    with pytest.raises(binding.MbertAttnError):
        binding.cross_attention(q, kv, kv, cq, ck, max_seqlen_q=-2 ** 32 + 3)


@pytest.mark.gpu
def test_amplitude_beyond_fp32(built):
    """The kernel holds it in fp32, where 1e39 is infinite."""
    x = torch.ones(1, 1, 64, device="cuda")
    p = torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(binding.MbertAttnError):
        binding.rotary(x, binding.Rotary(64, scaling={"kind": "yarn", "factor": 2.0, "original": 64,
                                                      "amplitude": 1e39}), positions=p)
    rope = binding.Rotary(64)
    rope.spec.amplitude = 3e38
    y = binding.rotary(x, rope, positions=p)
    assert (y == ctypes.c_float(3e38).value).all()
