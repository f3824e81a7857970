"""mbert_attn_get_error after calls on several streams: what any of them has
found is reported, once, by the first call that asks."""
import pytest
import torch

from encoder_only_transformer_gb300 import binding


@pytest.fixture(scope="module")
def built():
    import __graft_entry__
    __graft_entry__.build()


def offsets(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def calls():
    """(name, a call with bad offsets, the same with good ones)"""
    q = torch.randn(3, 2, 64, device="cuda").bfloat16()
    kv = torch.randn(10, 2, 64, device="cuda").bfloat16()
    qkv = torch.randn(10, 2304, device="cuda").bfloat16()
    rope = binding.Rotary(64)
    cq, good, bad = offsets(0, 3), offsets(0, 10), offsets(0, 11)
    return [
        ("cross", lambda cu: binding.cross_attention(q, kv, kv, cq, cu), bad, good),
        ("tokens", lambda cu: binding.cross_attention(q, kv, kv, cq, cu, max_seqlen_q=3), bad, good),
        ("rotary", lambda cu: binding.rotary(kv, rope, cu_seqlens=cu), bad, good),
        ("block", lambda cu: binding.attention(qkv, cu, "global"), offsets(0, 8, 5, 10), offsets(0, 5, 8, 10)),
    ]


@pytest.mark.gpu
@pytest.mark.parametrize("which", range(4), ids=["cross", "tokens", "rotary", "block"])
def test_error_on_another_stream_than_the_last(built, which):
    _, call, bad, good = calls()[which]
    h = binding._default(torch.device("cuda", 0))
    call(good)
    assert h.get_error() == 0
    late, last = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(late):
        torch.cuda._sleep(100_000_000)          # about 50 ms
        call(bad)
    if which != 3:                              # (the block's scratch is one call's at a time)
        with torch.cuda.stream(last):
            call(good)
    else:
        with torch.cuda.stream(last):
            binding.rotary(torch.ones(1, 1, 64, device="cuda"), binding.Rotary(64), cu_seqlens=offsets(0, 1))
    assert h.get_error() == -4
    assert h.get_error() == 0


@pytest.mark.gpu
def test_error_of_a_replayed_graph(built):
    """A replay goes past the handle: its errors are reported all the same."""
    _, call, bad, good = calls()[0]
    h = binding._default(torch.device("cuda", 0))
    cu = good.clone()
    call(cu)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        call(cu)
    assert h.get_error() == 0
    cu.copy_(bad)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
        graph.replay()
    assert h.get_error() == -4
    cu.copy_(good)
    graph.replay()
    assert h.get_error() == 0
