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


TILED = [  # T, K, N, G, act, res: enough rows and tokens for the tiles of 128 x 128
    (300, 64, 8300, 32, "bf16", "f32"), (300, 192, 8300, 32, "f16", "bf16"), (1000, 1152, 2700, 32, "bf16", "f16"),
    (130, 576, 16000, 64, "bf16", "f32"), (385, 640, 4200, 128, "f16", "f16"), (64, 128, 32000, 64, "f16", "f32"),
    (40, 320, 30001, 64, "bf16", "bf16"), (129, 1152, 12800, 128, "bf16", "f32"),
]


@pytest.mark.parametrize("T,K,N,G,act,res", TILED, ids=lambda v: str(v))
def test_tiles_exact_integers_and_random(T, K, N, G, act, res):
    import numpy as np
    import torch
    from oracle import linear_oracle as lo
    from test_gpu_linear import HALF_STEP, dt, make, run
    rng = np.random.default_rng(T * 131 + K + N)
    q = rng.integers(0, 16, (N, K))
    s = rng.integers(1, 4, (N, K // G)).astype(np.float16)
    b = rng.integers(-20, 4, (N, K // G)).astype(np.float16)
    x = rng.integers(-2, 3, (T, K)).astype(np.float32)
    got = run(make(K, N, G, act, q, s, b), torch.from_numpy(x).cuda().to(dt(act)), res, pad=2)
    want = torch.from_numpy(lo.linear(x, q, s, b, G)).to(dt(res)).double().numpy()
    assert np.array_equal(got, want)
    s = (rng.uniform(0.2, 1.2, (N, K // G)) / 40).astype(np.float16)
    b = (-7.5 * s * rng.uniform(0.8, 1.2, s.shape)).astype(np.float16)
    xr = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)).cuda().to(dt(act))
    x64 = xr.double().cpu().numpy()
    got = run(make(K, N, G, act, q, s, b), xr, res)
    ref, tol = lo.linear(x64, q, s, b, G), lo.error_bound(x64, q, s, b, G)
    tol = tol + HALF_STEP[res] * (np.abs(ref) + tol) + 2.0 ** -25   # the last term: half a step of fp16 subnormals
    assert (np.abs(got - ref) <= tol).all()


@pytest.mark.parametrize("G", [32, 64])
def test_nonfinite_tokens_of_a_tile_reach_their_own_row_only(G):
    import numpy as np
    import torch
    from test_gpu_linear import make, run
    rng = np.random.default_rng(4)
    K, N, T = 256, 200, 16500
    s = np.full((N, K // G), 0.01, np.float16)
    lin = make(K, N, G, "bf16", rng.integers(0, 16, (N, K)), s, (-8 * s).astype(np.float16))
    x = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)).cuda().bfloat16()
    clean = run(lin, x, "f32")
    x[7, 3], x[T - 1, 0] = float("nan"), float("inf")
    got = run(lin, x, "f32")
    assert np.isnan(got[7]).all() and not np.isfinite(got[T - 1]).any()
    keep = [t for t in range(T) if t not in (7, T - 1)]
    assert np.array_equal(got[keep], clean[keep])


@pytest.mark.parametrize("T,N,G", [(3, 70, 128), (3, 70, 32), (300, 9000, 128), (300, 9000, 32)])
def test_large_activations_whose_parts_cancel(T, N, G):
    # 512 |x| (1 + 16 s + |b|) is just within fp32's range; the two parts of a
    # group's sum are 30 times the result and more
    import numpy as np
    import torch
    from oracle import linear_oracle as lo
    from test_gpu_linear import make, run
    K = 1024
    rng = np.random.default_rng(N)
    q = 7 + (np.arange(K) + np.arange(N)[:, None]) % 2
    s, b = np.full((N, K // G), 0.01, np.float16), np.full((N, K // G), -0.075, np.float16)
    x = torch.from_numpy(5e35 * (1 - 0.2 * rng.random((T, K)))).float().cuda().bfloat16()
    x64 = x.double().cpu().numpy()
    assert 512 * np.abs(x64).max() * (1 + 0.16 + 0.075) < 3.4e38
    got = run(make(K, N, G, "bf16", q, s, b), x, "f32")
    ref, tol = lo.linear(x64, q, s, b, G), lo.error_bound(x64, q, s, b, G)
    assert (np.abs(got - ref) <= tol + 2.0 ** -24 * (np.abs(ref) + tol)).all()
