"""GPU int4 linear products: weights and outputs beyond one launch's reach."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K,N,G", [(2048, 70001, 32), (16384, 131103, 128)])
def test_more_packed_words_than_one_grid_dimension(K, N, G):
    # rows of a weight read out by unit vectors: whole numbers, exact in every
    # type; the scales lie behind the last values
    import torch
    from int4_routed_expert_router_amd import api
    g = torch.Generator(device="cuda").manual_seed(N)
    words = torch.randint(-2 ** 31, 2 ** 31, (N, K // 8), generator=g, device="cuda").to(torch.int32)
    s = torch.randint(1, 4, (N, K // G), generator=g, device="cuda").half()
    b = torch.randint(-8, 9, (N, K // G), generator=g, device="cuda").half()
    lin = api.Linear(K, N, G, words, s, b, act_dtype="f16")
    at = [0, 63, 1000, 1337, K - 1]
    x = torch.zeros(len(at), K, dtype=torch.float16, device="cuda")
    for t, k in enumerate(at):
        x[t, k] = 1
    y = torch.empty(len(at), N, device="cuda")
    api.linear(lin, x, y)
    torch.cuda.synchronize()
    for t, k in enumerate(at):
        q = (words[:, k // 8] >> (4 * (k % 8))) & 15
        assert torch.equal(y[t], q * s[:, k // G].float() + b[:, k // G].float())
