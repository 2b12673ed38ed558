"""GPU int4 linear product (moe_linear_pack, moe_linear_forward) against the
fp64 oracle: exact where every sum is exact, within the derived fp32 bound plus
the output's rounding otherwise."""
import numpy as np
import pytest

from oracle import linear_oracle as lo

pytestmark = pytest.mark.gpu

HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def dt(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def make(K, N, G, act, q, s, b):
    import torch
    from int4_routed_expert_router_amd import api
    return api.Linear(K, N, G, torch.from_numpy(lo.pack_words(q)).cuda(), torch.from_numpy(s).cuda(),
                      torch.from_numpy(b).cuda(), act_dtype=act)


def run(lin, x, res, pad=0):
    import torch
    from int4_routed_expert_router_amd import api
    T = x.shape[0]
    buf = torch.full((T + pad, lin.out_dim), 7.0, dtype=dt(res), device="cuda")
    api.linear(lin, x, buf[:T])
    torch.cuda.synchronize()
    assert (buf[T:] == 7.0).all()
    return buf[:T].double().cpu().numpy()


CASES = [  # T, K, N, G, act, res
    (1, 64, 1, 32, "bf16", "f32"), (1, 64, 33, 64, "f16", "f32"), (1, 2048, 1000, 64, "bf16", "bf16"),
    (2, 128, 31, 128, "f16", "f16"), (3, 576, 65, 64, "bf16", "f32"), (15, 640, 100, 32, "f16", "f32"),
    (16, 1024, 64, 128, "bf16", "f32"), (17, 320, 96, 64, "f16", "bf16"), (32, 448, 5, 32, "bf16", "f16"),
    (33, 8192, 129, 64, "bf16", "f32"), (64, 1024, 257, 128, "f16", "f32"), (65, 512, 48, 64, "bf16", "f32"),
    (127, 384, 160, 128, "bf16", "f32"), (129, 640, 130, 128, "f16", "f32"), (300, 1088, 259, 64, "bf16", "bf16"),
    (513, 2048, 385, 32, "f16", "f32"), (1000, 128, 128, 64, "bf16", "f32"),
    # many rows: the tiles of 128 tokens x 128 rows
    (70, 192, 16400, 64, "bf16", "f32"), (257, 64, 5600, 32, "f16", "f16"), (130, 640, 8300, 128, "f16", "f32"),
    (385, 320, 4200, 32, "bf16", "bf16"), (128, 1152, 16385, 128, "bf16", "f32"), (65, 576, 16300, 64, "f16", "f32"),
    (49, 128, 65440, 64, "f16", "bf16"), (64, 64, 65500, 32, "bf16", "f32"),
]
IDS = ["T%d_K%d_N%d_G%d_%s_%s" % c for c in CASES]


@pytest.mark.parametrize("T,K,N,G,act,res", CASES, ids=IDS)
def test_exact_integers(T, K, N, G, act, res):
    # small whole x, scales and biases: every product and sum is exact, so the
    # fp32 result is the exact one, rounded once to the output's type
    import torch
    rng = np.random.default_rng(T * 131 + K + N)
    q = rng.integers(0, 16, (N, K))
    s = rng.integers(1, 4, (N, K // G)).astype(np.float16)
    b = rng.integers(-20, 4, (N, K // G)).astype(np.float16)
    x = rng.integers(-2, 3, (T, K)).astype(np.float32)
    assert (np.abs(x) @ np.repeat(np.abs(s) * 32 + np.abs(b), G, 1).T.astype(np.float64)).max() < 2 ** 20
    lin = make(K, N, G, act, q, s, b)
    got = run(lin, torch.from_numpy(x).cuda().to(dt(act)), res, pad=2)
    want = torch.from_numpy(lo.linear(x, q, s, b, G)).to(dt(res)).double().numpy()
    assert np.array_equal(got, want)


@pytest.mark.parametrize("T,K,N,G,act,res", CASES, ids=IDS)
def test_random(T, K, N, G, act, res):
    import torch
    rng = np.random.default_rng(T * 137 + K + N)
    q = rng.integers(0, 16, (N, K))
    s = (rng.uniform(0.2, 1.2, (N, K // G)) / 40).astype(np.float16)
    b = (-7.5 * s * rng.uniform(0.8, 1.2, s.shape)).astype(np.float16)
    x = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)).cuda().to(dt(act))
    x64 = x.double().cpu().numpy()
    got = run(make(K, N, G, act, q, s, b), x, res)
    ref = lo.linear(x64, q, s, b, G)
    tol = lo.error_bound(x64, q, s, b, G)
    tol = tol + HALF_STEP[res] * (np.abs(ref) + tol) + 2.0 ** -25   # the last term: half a step of fp16 subnormals
    err = np.abs(got - ref)
    assert (err <= tol).all(), f"worst {float((err / tol).max()):.3f} of the bound"


def test_signed_and_zero_scales_and_full_range_values():
    import torch
    rng = np.random.default_rng(3)
    K, N, G, T = 256, 70, 32, 9
    q = rng.integers(0, 16, (N, K))
    q[:8] = 0
    q[8:16] = 15
    s = rng.standard_normal((N, K // G)).astype(np.float16)
    s[16:24] = 0
    b = (100 * rng.standard_normal((N, K // G))).astype(np.float16)
    s[24], b[24] = 0, 0
    for act, big in (("bf16", 1e30), ("f16", 6e4)):
        x = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)).cuda()
        x[1] *= big / 8
        x[2] *= 1e-6
        x[3] = 0
        x = x.clamp(-big, big).to(dt(act))
        x64 = x.double().cpu().numpy()
        got = run(make(K, N, G, act, q, s, b), x, "f32")
        assert (np.abs(got - lo.linear(x64, q, s, b, G)) <= 1.001 * lo.error_bound(x64, q, s, b, G)
                + 1e-37).all()
        assert (got[3] == 0).all() and (got[:, 24] == 0).all()


def test_nonfinite_tokens_reach_their_own_row_only():
    import torch
    rng = np.random.default_rng(4)
    K, N, G = 256, 40, 64
    q = rng.integers(0, 16, (N, K))
    s = np.full((N, K // G), 0.01, np.float16)
    lin = make(K, N, G, "bf16", q, s, (-8 * s).astype(np.float16))
    for T in (20, 200, 16500):
        x = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)).cuda().bfloat16()
        clean = run(lin, x, "f32")
        x[7, 3], x[T - 1, 0] = float("nan"), float("inf")
        got = run(lin, x, "f32")
        assert np.isnan(got[7]).all() and not np.isfinite(got[T - 1]).any()
        keep = [t for t in range(T) if t not in (7, T - 1)]
        assert np.array_equal(got[keep], clean[keep])


@pytest.mark.parametrize("T", [1, 40, 300, 9000])
def test_repeatable_captured_and_on_another_stream(T):
    import torch
    from int4_routed_expert_router_amd import api
    rng = np.random.default_rng(T)
    K, N, G = 1024, 192, 64
    q = rng.integers(0, 16, (N, K))
    s = rng.uniform(0.01, 0.02, (N, K // G)).astype(np.float16)
    lin = make(K, N, G, "bf16", q, s, (-7 * s).astype(np.float16))
    x = torch.randn(T, K, device="cuda").bfloat16()
    y = [torch.empty(T, N, device="cuda") for _ in range(3)]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    api.linear(lin, x, y[0], stream=st)
    st.synchronize()
    api.linear(lin, x, y[1])
    torch.cuda.synchronize()
    assert torch.equal(y[0], y[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.linear(lin, x, y[2])
    for i in range(4):
        x.copy_(torch.randn(T, K, device="cuda"))
        g.replay()
        api.linear(lin, x, y[1])
        torch.cuda.synchronize()
        assert torch.equal(y[1], y[2])


def test_packed_weights_hold_the_documented_bytes():
    import torch
    rng = np.random.default_rng(8)
    K, N, G = 192, 45, 64
    q = rng.integers(0, 16, (N, K))
    s = rng.standard_normal((N, 3)).astype(np.float16)
    b = rng.standard_normal((N, 3)).astype(np.float16)
    lin = make(K, N, G, "f16", q, s, b)
    torch.cuda.synchronize()
    got = lin.packed.cpu().numpy()
    rows = 64
    assert got.size == rows * K // 2 + 4 * rows * 3
    for _ in range(2000):
        r, k = int(rng.integers(rows)), int(rng.integers(K))
        p, tile, n = r // 32, (r // 16) % 2, r % 16
        c, ks, kb, j = k // 64, (k // 32) % 2, (k // 8) % 4, k % 8
        byte = (p * 3 + c) * 1024 + 16 * (16 * kb + n) + 4 * (2 * tile + ks)
        word = int(got[byte:byte + 4].view(np.uint32)[0])
        assert (word >> (4 * ((j >> 1) + 4 * (j & 1)))) & 15 == (q[r, k] if r < N else 0)
        at = rows * K // 2 + ((p * 3 + c) * 16 + n) * 8 + 4 * tile
        pair = got[at:at + 4].view(np.float16)
        assert np.array_equal(pair, [s[r, c], b[r, c]] if r < N else [0, 0])


def test_zero_tokens():
    import torch
    from int4_routed_expert_router_amd import api
    lin = make(64, 8, 64, "f16", np.zeros((8, 64), int), np.ones((8, 1), np.float16), np.ones((8, 1), np.float16))
    y = torch.full((0, 8), 3.0, device="cuda")
    api.linear(lin, torch.zeros(0, 64, dtype=torch.float16, device="cuda"), y)
    torch.cuda.synchronize()
