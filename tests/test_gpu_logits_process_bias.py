"""Long bias lists in which tokens stand more than once: the sums in list order, beside
every other option, and a time that grows with the list and not with its square."""
import numpy as np
import pytest
import torch

from tests import ref_answer as ref
from tests.test_gpu_logits_process import call, case, check, ragged

pytestmark = pytest.mark.gpu


def many(rng, V, n, distinct):
    """n biases on `distinct` tokens, the first and last of the vocabulary among them."""
    tokens = np.concatenate([[0, V - 1], rng.integers(0, V, max(distinct - 2, 0))])
    return [(int(v), float(np.float32(b))) for v, b in zip(rng.choice(tokens, n), rng.normal(size=n) * 5)]


@pytest.mark.parametrize("V,n,distinct", [(40, 700, 9), (5000, 513, 400), (5000, 3000, 1), (50001, 4000, 1500),
                                          (290003, 2500, 2000)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_repeated_tokens_in_long_lists(gpu_lib, V, n, distinct, dtype):
    rng = np.random.default_rng(n + V)
    vals, dev, kw = case(4, V, V, dtype, n_prompt=300, n_output=200)
    kw["bias"][0], kw["bias"][2] = many(rng, V, n, distinct), many(rng, V, n + 31, distinct)
    kw["bias"][2][::50] = [(-1, 3.0), (V, 2.0)] * (len(kw["bias"][2][::50]) // 2) + [(V + 5, 1.0)] * (len(kw["bias"][2][::50]) % 2)
    kw["mask"][0], kw["mask"][2] = rng.random(V) < 0.5, True
    # half of them also in the row's other lists
    kw["output"][0] += [v for v, _ in kw["bias"][0][:150]]
    kw["prompt"][2] += [v for v, _ in kw["bias"][2][:150] if 0 <= v < V]
    check(call(gpu_lib, dev, kw), vals, kw)


@pytest.mark.parametrize("V", [50001, 270001])
def test_beside_long_token_lists(gpu_lib, V):
    """Clusters of blocks, and columns computed in several rounds."""
    rng = np.random.default_rng(V)
    vals, dev, kw = case(3, V, 23, torch.float32, n_prompt=70000, n_output=50000)
    kw["output"][1] = rng.integers(0, V, 40000).tolist()
    for t in range(3):
        kw["bias"][t] = many(rng, V, 1500, 900) + [(v, 0.25) for v in kw["output"][t][:600]] * 2
    check(call(gpu_lib, dev, kw), vals, kw)


@pytest.mark.parametrize("n", [300, 2000])
def test_sums_are_taken_in_list_order(gpu_lib, n):
    """Bitwise the fp32 sums of the list, one entry after the other."""
    V, T = 3001, 3
    rng = np.random.default_rng(n)
    z = rng.standard_normal((T, V)).astype(np.float32)
    lists = [rng.integers(0, 40, n) * 70 for _ in range(T)]
    values = [(rng.normal(size=n) * 10.0 ** rng.integers(-6, 7, n)).astype(np.float32) for _ in range(T)]
    tokens, offsets = ragged([x.tolist() for x in lists])
    got = gpu_lib.logits_process_f32(torch.from_numpy(z).cuda(), bias_tokens=tokens, bias_offsets=offsets,
                                     bias=torch.from_numpy(np.concatenate(values)).cuda()).cpu().numpy()
    for t in range(T):
        add = {}
        for v, b in zip(lists[t], values[t]):
            add[v] = b if v not in add else np.float32(add[v] + b)
        want = z[t].copy()
        for v, b in add.items():
            want[v] = np.float32(want[v] + b)
        assert (got[t] == want).all()


def test_time_grows_with_the_list(gpu_lib):
    """60000 biases, one or all of them twice in the list: a search for every entry's
    repetitions is 3.6e9 steps."""
    V, n = 128256, 60000
    rng = np.random.default_rng(1)
    z = torch.from_numpy(rng.standard_normal((1, V)).astype(np.float32)).cuda()
    offsets = torch.tensor([0, n], device="cuda")
    bias = torch.from_numpy(rng.normal(size=n).astype(np.float32)).cuda()
    once = rng.permutation(V)[:n]
    one_twice, all_twice = once.copy(), np.concatenate([once[:n // 2], once[:n // 2][::-1]])
    one_twice[n - 1] = once[0]
    out = torch.empty((1, V), device="cuda")
    for tokens in (one_twice, all_twice):
        ids = torch.from_numpy(tokens).cuda()

        def run():
            gpu_lib.logits_process_f32(z, bias_tokens=ids, bias=bias, bias_offsets=offsets, out=out)
        run()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        run()
        b.record()
        torch.cuda.synchronize()
        ms = a.elapsed_time(b)
        print(f"{ms:.3f} ms")
        vals = z.double().cpu().numpy()
        want, bound = ref.process(vals, bias=[list(zip(tokens.tolist(), bias.double().cpu().tolist()))])
        assert (np.abs(out.double().cpu().numpy() - want) <= 4 * ref.U24 * (np.abs(vals) + np.abs(want - vals) + 8)).all()
        assert ms < 10
