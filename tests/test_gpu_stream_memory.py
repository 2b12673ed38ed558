"""Memory that the binding allocates for a call on another stream comes from that
stream's blocks: a block just freed on the current stream, which work waiting
there may still read, is not taken."""
import pytest

pytestmark = pytest.mark.gpu


def freed_block(nbytes):
    """Address of a block of the current stream's that has just been freed."""
    import torch
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    t = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    at = t.data_ptr()
    del t
    # without another stream in play it is the next one handed out
    again = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    assert again.data_ptr() == at
    del again
    return at


def test_workspace_of_the_layer_calls():
    import synth
    import torch
    from int4_routed_expert_router_amd import api
    from moe_testlib import desc_for
    desc, s = desc_for(synth.TINY), torch.cuda.Stream()
    at = freed_block(max(api.workspace_bytes(desc, 5), 256))
    assert api._scratch(desc, 5, torch.device("cuda", 0), None).data_ptr() == at
    assert api._scratch(desc, 5, torch.device("cuda", 0), torch.cuda.current_stream()).data_ptr() == at
    assert api._scratch(desc, 5, torch.device("cuda", 0), s).data_ptr() != at


def test_workspace_of_gdn_prefill(monkeypatch):
    import torch
    from int4_routed_expert_router_amd import api
    seen = []
    make = api.gdn_prefill_workspace
    monkeypatch.setattr(api, "gdn_prefill_workspace", lambda *a, **k: seen.append(make(*a, **k)) or seen[-1])
    q, v = torch.randn(90, 1, 128, device="cuda").bfloat16(), torch.randn(90, 2, 16, device="cuda").bfloat16()
    g, beta = -torch.rand(90, 2, device="cuda"), torch.rand(90, 2, device="cuda")
    off = torch.tensor([0, 90], dtype=torch.int32, device="cuda")
    outs = []
    for stream in (None, torch.cuda.Stream()):
        state, o = torch.zeros(1, 2, 16, 128, device="cuda"), torch.empty(90, 2, 16, device="cuda")
        n = make(1, 90, 1, 2, 16).numel()
        at = freed_block(n)
        api.gdn_prefill(q, q, v, g, beta, state, o, off, 0.1, stream=stream)
        torch.cuda.synchronize()
        assert (seen[-1].data_ptr() == at) == (stream is None)
        outs.append((o, state))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
def test_packed_weights(raw):
    import torch
    from int4_routed_expert_router_amd import api
    K, N = 1024, 4096
    words = torch.randint(-2 ** 31, 2 ** 31, (N, K // 8), device="cuda").to(torch.int32)
    sc = torch.rand(N, K // 64, device="cuda").half()
    x = torch.randn(3, K, device="cuda").bfloat16()
    s = torch.cuda.Stream()
    n = int(api.lib().moe_linear_bytes(K, N, 64))
    y = [torch.empty(3, N, device="cuda") for _ in range(2)]
    api.linear(api.Linear(K, N, 64, words, sc, -sc), x, y[0])
    at = freed_block(n)
    lin = api.Linear(K, N, 64, words, sc, -sc, stream=s.cuda_stream if raw else s)
    assert lin.packed.data_ptr() != at
    s.synchronize()
    api.linear(lin, x, y[1])
    torch.cuda.synchronize()
    assert torch.equal(y[0], y[1])
