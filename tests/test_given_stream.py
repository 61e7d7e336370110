"""A call that is given a stream allocates, fills and copies under that stream, not
under the current one: host-side check of every such call with a fake library (no GPU),
and the results of calls beside a delayed current stream (GPU)."""
import contextlib
import inspect

import pytest
import torch

import lm_head_online_gb300 as lmho

HANDLE = 0x1234560


class Stream:
    cuda_stream = HANDLE


class Library:
    """Sizes of 256 bytes; calls succeed and note their last argument, the stream."""

    def __init__(self):
        self.streams = []

    def __getattr__(self, name):
        if name.endswith("workspace_bytes"):
            return lambda *a: 256

        def call(*a):
            self.streams.append(a[-1])
            return 0
        return call


def i64(*shape):
    return torch.zeros(shape, dtype=torch.int64)


def f32(*shape):
    return torch.zeros(shape)


def b16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


T, H, V, S, B = 4, 8, 16, 2, 2
HEADS = dict(xs=b16(T, H), Ws=b16(V, H), xt=b16(T, H), Wt=b16(V, H))
SHARDS = dict(xs=b16(T, H), Ws_local=b16(V, H), xt=b16(T, H), Wt_local=b16(V, H))
CALLS = {
    "ce_fwd_f32": dict(logits=f32(T, V), target=i64(T)),
    "ce_fwd_sbv_bf16": dict(logits=b16(S, B, V), target=i64(S, B)),
    "ce_partials_sbv_bf16": dict(logits_local=b16(S, B, V), target=i64(S, B), vocab_start=0),
    "ce_partials_f32": dict(logits_local=f32(T, V), target=i64(T), vocab_start=0),
    "ce_merge_partials": dict(partials=f32(2, 3, S, B), target=i64(S, B), V=V),
    "ce_fwd_bwd_f32": dict(logits=f32(T, V), target=i64(T)),
    "ce_fwd_bwd_sbv_bf16": dict(logits=b16(S, B, V), target=i64(S, B)),
    "flce_fwd_bf16": dict(x=b16(T, H), W=b16(V, H), target=i64(T)),
    "flce_fwd_bwd_bf16": dict(x=b16(T, H), W=b16(V, H), target=i64(T)),
    "flce_cpo_fwd_bf16": dict(x=b16(B, S, H), W=b16(V, H), target=i64(B, S)),
    "flce_cpo_fwd_bwd_bf16": dict(x=b16(B, S, H), W=b16(V, H), target=i64(B, S)),
    "fljsd_fwd_bf16": HEADS,
    "fljsd_fwd_bf16_ex": HEADS,
    "fljsd_fwd_bwd_bf16": HEADS,
    "flce_partials_bf16": dict(x=b16(T, H), W_local=b16(V, H), target=i64(T), vocab_start=0),
    "flce_shard_bwd_bf16": dict(x=b16(T, H), W_local=b16(V, H), target=i64(T), partials=f32(2, 3, T), vocab_start=0, V=V),
    "cpo_combine_rows": dict(rows=f32(T), B=B),
    "fljsd_lse_partials_bf16": SHARDS,
    "lse_merge_partials": dict(parts=f32(2, 2, T)),
    "fljsd_terms_bf16": dict(SHARDS, lse=f32(2, T)),
    "fljsd_shard_bwd_bf16": dict(SHARDS, lse=f32(2, T), kl=f32(T)),
    "jsd_merge_terms": dict(terms=f32(2, T)),
    "rows_mean": dict(rows=f32(T)),
    "head_lora_bf16": dict(x=b16(T, H), W=b16(V, H), A=b16(1, 8, H), B=b16(1, V, 8), adapter=i64(T)),
    "logits_process_f32": dict(logits=f32(T, V)),
    "logits_process_bf16": dict(logits=b16(T, V)),
    "logits_choose_f32": dict(logits=f32(T, V), n=2),
    "logits_choose_bf16": dict(logits=b16(T, V), n=2),
    "workspace": dict(nbytes=256, device="cpu"),
}
OTHERS = {"ce_fwd_f32_noalloc", "copy_h2d", "ws_status", "selftest_wait_timeout",  # allocate nothing
          "probe_read"}                                                          # looks at its tensor itself


@pytest.fixture
def fake(monkeypatch):
    """The binding on CPU tensors with a fake library; .current = the current stream's
    handle, .made = that at every allocation."""
    lib = Library()
    lib.current, lib.made = 0, []

    @contextlib.contextmanager
    def stream(s):
        before, lib.current = lib.current, getattr(s, "cuda_stream", s)
        yield
        lib.current = before
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: handle)
    for name in ("empty", "empty_like", "zeros"):
        def made(*a, _real=getattr(torch, name), **kw):
            lib.made.append(lib.current)
            return _real(*a, **kw)
        monkeypatch.setattr(torch, name, made)
    monkeypatch.setattr(lmho, "load", lambda: lib)
    monkeypatch.setattr(lmho, "_dev", lambda t, *a: t.data_ptr())
    monkeypatch.setattr(lmho, "_host_or_dev", lambda t, *a: t.data_ptr())
    monkeypatch.setattr(lmho, "_on", lambda *a: contextlib.nullcontext())
    monkeypatch.setattr(lmho, "_cuda_device", lambda *a: torch.device("cpu"))
    return lib


def test_every_call_with_a_stream_is_listed():
    have = {n for n, f in vars(lmho).items() if inspect.isfunction(f) and not n.startswith("_")
            and "stream" in inspect.signature(f).parameters}
    assert have == set(CALLS) | OTHERS


@pytest.mark.parametrize("name", CALLS)
def test_allocations_are_made_under_the_given_stream(fake, name):
    getattr(lmho, name)(**CALLS[name], stream=Stream())
    assert fake.made and set(fake.made) == {HANDLE}
    assert fake.current == 0 and set(fake.streams) <= {HANDLE}
    fake.made.clear()
    fake.streams.clear()
    getattr(lmho, name)(**CALLS[name], stream=HANDLE)         # a bare handle
    assert fake.made and set(fake.made) == {HANDLE} and set(fake.streams) <= {HANDLE}


@pytest.mark.gpu
@pytest.mark.parametrize("bare", [False, True])
def test_results_beside_a_delayed_current_stream(gpu_lib, bare):
    """The current stream is held up for tens of milliseconds while calls on another
    stream make their own outputs and workspaces."""
    gen = torch.Generator(device="cuda").manual_seed(3)

    def normal(*shape):
        return torch.randn(shape, device="cuda", generator=gen).bfloat16()
    x, W, A, B_ = normal(300, 128), normal(2000, 128), normal(9, 16, 128), normal(9, 2000, 16)
    ids = torch.randint(-1, 9, (300,), device="cuda", generator=gen)
    target = torch.randint(0, 2000, (300,), device="cuda", generator=gen)
    mask = torch.randint(-2 ** 31, 2 ** 31 - 1, (300, 63), device="cuda", generator=gen).to(torch.int32)

    def calls(stream):
        z = gpu_lib.head_lora_bf16(x, W, A, B_, ids, stream=stream)
        y = gpu_lib.logits_process_f32(z, mask=mask, stream=stream)
        loss, dx, dW = gpu_lib.flce_fwd_bwd_bf16(x, W, target, stream=stream)
        return [z, y, *gpu_lib.logits_choose_f32(y, 20, stream=stream), loss, dx, dW]
    want = calls(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    handle = side.cuda_stream if bare else side
    for _ in range(3):
        torch.cuda._sleep(40_000_000)
        got = calls(handle)
        junk = [torch.full((1 << 20,), 7, device="cuda") for _ in range(8)]   # the current stream's, once it goes on
        side.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g, w)
        del junk
        torch.cuda.synchronize()


@pytest.mark.gpu
def test_the_default_stream_by_its_handle(gpu_lib):
    z = torch.randn(5, 300, device="cuda")
    want = gpu_lib.logits_choose_f32(z, 4)
    for handle in (0, torch.cuda.default_stream()):
        for g, w in zip(gpu_lib.logits_choose_f32(z, 4, stream=handle), want):
            assert torch.equal(g, w)
