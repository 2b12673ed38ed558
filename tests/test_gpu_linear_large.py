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


@pytest.mark.parametrize("T,N,G", [(16500, 40, 64), (128 * 128, 128, 32), (9001, 300, 128), (4999, 1157, 64),
                                   (700, 3001, 64), (130, 16385, 32)])
def test_tiles_of_any_count(T, N, G):
    # few and uneven row and token tiles; small whole numbers, exact in fp32
    import torch
    from int4_routed_expert_router_amd import api
    K = 128
    g = torch.Generator(device="cuda").manual_seed(T + N)
    words = torch.randint(-2 ** 31, 2 ** 31, (N, K // 8), generator=g, device="cuda").to(torch.int32)
    s = torch.randint(1, 4, (N, K // G), generator=g, device="cuda").half()
    b = torch.randint(-20, 4, (N, K // G), generator=g, device="cuda").half()
    x = torch.randint(-2, 3, (T, K), generator=g, device="cuda").bfloat16()
    y = torch.full((T + 3, N), 7.0, device="cuda")
    api.linear(api.Linear(K, N, G, words, s, b), x, y[:T])
    q = torch.stack([(words >> (4 * j)) & 15 for j in range(8)], -1).view(N, K)
    w = q * s.double().repeat_interleave(G, 1) + b.double().repeat_interleave(G, 1)
    assert torch.equal(y[:T].double(), x.double() @ w.t().contiguous()) and (y[T:] == 7.0).all()
