"""The head's adapters at the ends of the number range: x A^T past the largest bf16, and
infinite entries of B, against the definition in 64 bits."""
import numpy as np
import pytest
import torch

from tests import ref_answer as ref
from tests.test_gpu_head_lora import check, make

pytestmark = pytest.mark.gpu


def to_dev(values):
    got, bits = ref.bf16_values(values)
    return got, torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16).cuda()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,r", [(3, 8), (40, 24), (200, 40)])
def test_finite_h_past_the_largest_bf16(gpu_lib, T, r, dtype):
    """x A^T = 1 and a scale between bf16's largest number and fp32's."""
    H, V = 64, 300
    top = float(torch.finfo(torch.float32).max)
    rng = np.random.default_rng(r)
    x, dx = to_dev(np.eye(1, H).repeat(T, 0))
    W, dW = to_dev(np.zeros((V, H)))
    A, dA = to_dev(np.where(np.arange(r)[None, :, None] == 0, 1.0, 0.0).repeat(3, 0) * np.eye(1, H))
    B, dB = to_dev(rng.choice([-1.0, 1.0], (3, V, r)) * 2.0 ** rng.integers(-20, -2, (3, V, r)))
    scale = np.array([top, 3.4e38, -3.395e38], np.float32)
    ids = rng.integers(0, 3, T)
    got = gpu_lib.head_lora_bf16(dx, dW, dA, dB, torch.from_numpy(ids).cuda(), scale=torch.from_numpy(scale).cuda(),
                                 dtype=dtype).double().cpu().numpy()
    want = scale.astype(np.float64)[ids][:, None] * B[ids, :, 0]
    # three parts: all 24 bits, times a power of two, in sums that cut bits (16 steps);
    # bf16: 16 bits and the result's own rounding
    tol = 16 * ref.U24 if dtype == torch.float32 else ref.U8 + ref.U8 * ref.U8 + 16 * ref.U24
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= tol * np.abs(want)).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,V,r", [(1, 130, 8), (50, 301, 16), (33, 1000, 32), (300, 264, 40), (260, 517, 24)])
def test_infinite_entries_of_b(gpu_lib, T, V, r, dtype):
    """One infinite entry in a row of B makes that logit h's sign times it; the others stay."""
    H, n = 128, 5
    rng = np.random.default_rng(T + r)
    x, dx = to_dev(rng.standard_normal((T, H)))
    x[::3] = np.round(x[::3])                              # h of few bits: some parts are 0
    x, dx = to_dev(x)
    W, dW = to_dev(rng.standard_normal((V, H)) / 8)
    A, dA = to_dev(rng.integers(-4, 5, (n, r, H)))
    B, dB = to_dev(rng.standard_normal((n, V, r)))
    ids = rng.integers(-1, n, T)
    ids[0] = 2
    clean = gpu_lib.head_lora_bf16(dx, dW, dA, dB, torch.from_numpy(ids).cuda(), dtype=dtype)
    rank = rng.integers(0, r, V)
    sign = rng.choice([-1.0, 1.0], V)
    holds = rng.random(V) < 0.3
    holds[[0, V - 1]] = True
    for v in np.flatnonzero(holds):
        B[2, v, rank[v]] = sign[v] * np.inf
    _, dB = to_dev(B)
    got = gpu_lib.head_lora_bf16(dx, dW, dA, dB, torch.from_numpy(ids).cuda(), dtype=dtype)
    h = x @ A[2].T                                          # [T, r]
    mine = np.flatnonzero(ids == 2)
    assert (np.abs(h[mine]) > 1e-3).all() or (np.abs(h[mine])[np.abs(h[mine]) <= 1e-3] == 0).all()
    g, c = got.double().cpu().numpy(), clean.double().cpu().numpy()
    for t in range(T):
        if ids[t] != 2:
            assert (g[t] == c[t]).all()
            continue
        assert (g[t, ~holds] == c[t, ~holds]).all()
        hv = h[t, rank]
        with np.errstate(invalid="ignore"):
            want = hv * sign * np.inf                       # 0 inf is NaN
        assert np.array_equal(g[t, holds], want[holds], equal_nan=True)


@pytest.mark.parametrize("bad", [np.inf, -np.inf])
def test_infinite_h(gpu_lib, bad):
    """An infinite entry of A: the logit is its sign through x and B; B = 0 gives NaN."""
    T, H, V, r = 20, 64, 100, 16
    rng = np.random.default_rng(7)
    x, dx = to_dev(rng.choice([-1.0, 1.0], (T, H)) * rng.uniform(1, 2, (T, H)))
    W, dW = to_dev(rng.standard_normal((V, H)))
    A = np.zeros((1, r, H))
    A[0, 3, 5] = bad
    A, dA = to_dev(A)
    B, dB = to_dev(rng.choice([-1.0, 0.0, 1.0], (1, V, r)))
    for dtype in (torch.float32, torch.bfloat16):
        got = gpu_lib.head_lora_bf16(dx, dW, dA, dB, torch.zeros(T, dtype=torch.int64, device="cuda"), dtype=dtype)
        with np.errstate(invalid="ignore"):
            want = (x[:, 5] * bad)[:, None] * B[0, :, 3][None, :]
        assert np.array_equal(got.double().cpu().numpy(), want, equal_nan=True)


@pytest.mark.parametrize("T", [100, 300])
def test_several_units_repeat_and_stay_within_the_bound_in_any_order(gpu_lib, T):
    """Blocks with several units of a token tile: equal calls give equal bits; the tokens
    in another order may round differently, within the same bound."""
    vals, dev, adapter, scale = make(T, 512, 30011, 9, 16, seed=T)
    s, ids = torch.from_numpy(scale).cuda(), torch.from_numpy(adapter).cuda()
    got = gpu_lib.head_lora_bf16(*dev, ids, scale=s)
    check(got, vals, adapter, scale)
    assert torch.equal(gpu_lib.head_lora_bf16(*dev, ids, scale=s), got)
    order = torch.randperm(T, generator=torch.Generator().manual_seed(3)).cuda()
    mixed = gpu_lib.head_lora_bf16(dev[0][order].contiguous(), *dev[1:], ids[order].contiguous(), scale=s)
    check(mixed[torch.argsort(order)], vals, adapter, scale)
