"""Log-probabilities and tokens over the whole range of finite logits, each row held to
a bound of its own: fills that masks use, small temperatures, forced tokens, rows with
one live token."""
import numpy as np
import pytest
import torch

from tests import ref_answer as ref
from tests.test_gpu_logits_choose import call, to_dev

pytestmark = pytest.mark.gpu


def log_probs(z, tokens):
    """fp64 log-probabilities of `tokens` (-1: -inf) with the largest logit taken off first:
    z - (max + ln sum) has lost ln sum where 64 bits round the maximum by more."""
    out = np.full(tokens.shape, -np.inf)
    for t, row in enumerate(z.astype(np.float64)):
        m = row.max()
        if m == -np.inf:
            continue
        there = tokens[t] >= 0
        out[t, there] = (row[tokens[t, there]] - m) - np.log(np.exp(row - m).sum())
    return out


def check_rows(got, dev, n, **kw):
    """Tokens equal; a log-probability within its own rounding (z - max, the difference
    from ln sum: 4 u of it), the normaliser's (lse_bound) and that of the exponents
    (three roundings of z - max, weighted by the softmax: at most 3 u ln V) -- nothing
    that grows with the logits, and nothing of another row."""
    z = dev.float().cpu().numpy()
    V = z.shape[1]
    token, _, best, _, sure = ref.choose(z, n, **kw)
    logprob, best_lp = log_probs(z, token[:, None])[:, 0], log_probs(z, best)
    gt, glp, gb, gblp = (g.cpu().numpy().astype(np.float64) for g in got)
    assert (gb == best).all()
    assert sure.all() and (gt == token).all()

    def close(a, b):
        tol = ref.lse_bound(V) + 3 * ref.U24 * np.log(V) + 4 * ref.U24 * np.where(np.isfinite(b), np.abs(b), 0.0)
        with np.errstate(invalid="ignore"):
            return ((a == b) | (np.abs(a - b) <= tol)).all()
    assert not np.isnan(gblp).any() and close(gblp, best_lp)
    assert close(glp, logprob)


FILLS = [31.1, -1.0e4, 2000.3, 1.0e6, 1.2e7, 3.1e9, -1.0e9, 1.0e10, -1.0e10, 1.0e30, -1.0e30, 3.0e38, -3.0e38]


@pytest.mark.parametrize("V", [40, 1000, 40003])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_of_one_value(gpu_lib, V, dtype):
    """Every token has -ln V, whatever the value."""
    dev = to_dev(np.repeat(np.array(FILLS, np.float32)[:, None], V, 1), dtype)
    got = call(gpu_lib, dev, 9)
    check_rows(got, dev, 9)
    assert (got[0] == 0).all()


@pytest.mark.parametrize("V", [40, 1000, 40003])
@pytest.mark.parametrize("rest", [-np.inf, -3.4e38])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_one_live_token_has_probability_one(gpu_lib, V, rest, dtype):
    z = np.full((len(FILLS), V), rest, np.float32)
    at = np.arange(len(FILLS)) * (V - 1) // (len(FILLS) - 1)
    z[np.arange(len(FILLS)), at] = FILLS
    dev = to_dev(z, dtype)
    live = dev.float().amax(1) > -1e38                  # else the rest is as large
    got = call(gpu_lib, dev, 1)
    assert (got[0].cpu().numpy()[live.cpu()] == at[live.cpu()]).all()
    assert (got[1][live] == 0).all() and (got[3][live] == 0).all()


@pytest.mark.parametrize("V", [300, 5000, 40003])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_scaled_shifted_and_forced_rows(gpu_lib, V, dtype):
    rng = np.random.default_rng(V)
    body = rng.standard_normal((10, V)).astype(np.float32) * 3
    z = body.copy()
    z[0] *= 1e5                                          # temperatures of 1e-5 and 1e-9
    z[1] *= 1e9
    z[2] += 2.0e4                                        # far from 0
    z[3] -= 2.0e6
    z[4] += 1.2e7
    z[5, V // 2] += 1.0e9                                # a forced token
    z[6, rng.permutation(V)[:V - 7]] = -1.0e9            # fills of a mask, few allowed
    z[7, rng.permutation(V)[:V - 7]] = -1.0e30
    z[8, :V - 3] = -3.0e38
    z[9] = z[9] * 10 + 30
    dev = to_dev(z, dtype)
    for n in (1, 16, 128):
        check_rows(call(gpu_lib, dev, n), dev, n)
    noise = rng.gumbel(size=(10, 16)).astype(np.float32)
    top_k = np.full(10, 5, np.int64)
    check_rows(call(gpu_lib, dev, 16, noise=noise, top_k=top_k), dev, 16, noise=noise, top_k=top_k)


def test_small_temperature_and_bias_of_the_step_before(gpu_lib):
    """Rows as logits_process gives them: divided by 1e-8, or with a bias of 1e9."""
    rng = np.random.default_rng(4)
    z = to_dev(rng.standard_normal((4, 3000)) * 4, torch.float32)
    z[:, 77] = 20.0
    cold = gpu_lib.logits_process_f32(z, temperature=torch.full((4,), 1e-8, device="cuda"))
    forced = gpu_lib.logits_process_f32(z, bias_tokens=torch.full((4,), 5, device="cuda"),
                                        bias=torch.full((4,), 1e9, device="cuda"),
                                        bias_offsets=torch.arange(5, device="cuda"))
    for dev, want in ((cold, 77), (forced, 5)):
        got = call(gpu_lib, dev, 3)
        check_rows(got, dev, 3)
        assert (got[0] == want).all() and (got[1] == 0).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_non_finite_rows_beside_large_ones(gpu_lib, dtype):
    """The masked, empty and non-finite rows, each finite one held to its own bound."""
    rng = np.random.default_rng(1)
    V, n = 9000, 12
    z = rng.standard_normal((8, V)).astype(np.float32)
    z[0] = -np.inf
    z[1, 1:] = -np.inf
    z[2, 8999] = np.nan
    z[3, 17] = np.inf
    z[4, :8995] = -np.inf
    z[5] = -3.0e38
    z[6, ::2] = -3.0e38
    dev = to_dev(z, dtype)
    finite = [0, 1, 4, 5, 6, 7]
    got = call(gpu_lib, dev, n)
    check_rows([g[finite] for g in got], dev[finite], n)
    for row in (2, 3):
        assert got[0][row] == -1 and torch.isnan(got[1][row]) and torch.isnan(got[3][row]).all()
