"""What the cache and scoring calls do on the host around the library: the
workspaces, streams and devices they pass, and the calls they refuse.  CPU only:
a stand-in for the library records what reaches it, CPU tensors stand for device
tensors."""
import contextlib
import gc
import threading
import types
import weakref

import pytest
import torch

from test_binding_checks import cs
from test_cache_score_checks import (FAKE, I3, INVALID, UNSUPPORTED, attend as c_attend, cache as fake_cache, evict,
                                     grad, score)

from commit_step_gb300 import cache as cache_mod
from commit_step_gb300 import score as score_mod

STREAM = 77


class FakeLib:
    """Records the calls; everything succeeds.  Sizes come from the library."""

    def __init__(self):
        self.calls = []
        self.attend_hook = lambda: None

    def __getattr__(self, name):
        if name.endswith("_workspace_size"):
            return getattr(cs.lib_handle(), name)

        def call(*args):
            self.calls.append((name, args))
            if name == "dllm_cache_attention":
                self.attend_hook()
            return 0

        return call

    def workspaces(self):
        """(address, bytes) of each attention's workspace."""
        return [(a[16], a[17]) for name, a in self.calls if name == "dllm_cache_attention"]


@pytest.fixture
def lib(monkeypatch):
    fake = FakeLib()
    monkeypatch.setattr(cache_mod, "_lib", fake)
    monkeypatch.setattr(cache_mod, "_raw_stream", lambda stream, index: STREAM)
    monkeypatch.setattr(cache_mod, "_need_cuda", lambda *ts: None)
    monkeypatch.setattr(cache_mod, "_NEED", {})
    monkeypatch.setattr(cache_mod, "_KEPT", threading.local(), raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: None)
    monkeypatch.setattr(torch.cuda, "stream", lambda stream: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    return fake


def host_cache(pages=8, page_size=16, heads=4, dim=64):
    codes = torch.zeros((pages, heads, page_size, dim), dtype=torch.uint8)
    scale = torch.ones((pages, heads))
    return cs.KVCache.from_tensors(codes, codes.clone(), scale, scale.clone())


def attend(cache, B, L, Hq, **kw):
    q = torch.zeros((B, L, Hq, cache.head_dim), dtype=torch.bfloat16)
    table = torch.zeros((B, 2), dtype=torch.int32)
    return cs.cache_attention(q, cache, table, torch.zeros(B, dtype=torch.int32), **kw)


def need(cache, B, L, Hq):
    return int(cs.lib_handle().dllm_cache_attention_workspace_size(B, L, Hq, cache.heads, cache.head_dim))


@pytest.mark.parametrize("before,after", [((0, 32, 8), (2, 32, 8)), ((2, 13, 10), (2, 8, 16)), ((2, 0, 8), (1, 1, 4))])
def test_the_workspace_of_a_call_does_not_go_by_an_empty_or_refused_one(lib, before, after):
    """An empty batch; heads that do not divide (13 x 10 and 8 x 16 queries give as
    many rows of a key head, rounded down); no queries."""
    cache = host_cache()
    attend(cache, *before)
    attend(cache, *after)
    assert lib.workspaces()[-1][1] >= need(cache, *after)


def test_two_threads_on_one_stream_do_not_share_a_workspace(lib):
    """The calls overlap (ctypes lets go of the interpreter's lock), and a call's
    later launches read what its first one left in the workspace."""
    cache, both = host_cache(), threading.Barrier(2, timeout=20)
    lib.attend_hook = both.wait
    threads = [threading.Thread(target=attend, args=(cache, 2, 32, 8)) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    a, b = lib.workspaces()
    assert a[0] + a[1] <= b[0] or b[0] + b[1] <= a[0]


class Streams:
    """Stands for torch.cuda's current stream: which it is, and whether it is being captured."""

    def __init__(self, monkeypatch):
        self.current, self.captured = 1, set()
        monkeypatch.setattr(torch.cuda, "stream", self.enter)
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: self.current in self.captured)
        monkeypatch.setattr(cache_mod, "_raw_stream", lambda stream, index: self.current if stream is None else stream)

    @contextlib.contextmanager
    def enter(self, stream):
        before, self.current = self.current, stream
        yield
        self.current = before


@pytest.mark.parametrize("given", [False, True])
def test_a_captured_call_has_a_workspace_of_its_own(lib, monkeypatch, given):
    """A graph keeps addresses: not that of a workspace which a later call may
    replace; and its own memory is not kept for calls outside of it.  The stream
    that counts is the one the call runs on."""
    streams, made, empty = Streams(monkeypatch), [], cache_mod._empty

    def recorded(shape, dtype, device, stream):
        t = empty(shape, dtype, device, stream)
        if dtype == torch.uint8:
            made.append((t.data_ptr(), weakref.ref(t)))
        return t

    monkeypatch.setattr(cache_mod, "_empty", recorded)
    cache = host_cache()

    def call(L):
        if given:
            attend(cache, 2, L, 8, stream=2)
        else:
            with streams.enter(2):
                attend(cache, 2, L, 8)

    call(32)                                   # the warm-up
    streams.captured = {2}
    call(4)
    call(16)
    streams.captured = {1}                     # (another stream's capture does not matter)
    call(4)
    gc.collect()
    assert len(made) == 3 and made[0][1]() is not None
    assert made[1][1]() is None and made[2][1]() is None
    at = [a for a, _ in lib.workspaces()]
    assert at[0] == at[3] == made[0][0] and at[0] not in at[1:3]


@pytest.mark.parametrize("current,stream_on", [(1, None), (-1, 1)])
def test_another_device_is_refused(monkeypatch, current, stream_on):
    """The tensors' device (-1 here) is not the current one, or not the stream's:
    nothing reaches the library."""
    fake = FakeLib()
    for mod in (cache_mod, score_mod):
        monkeypatch.setattr(mod, "_lib", fake)
        monkeypatch.setattr(mod, "_need_cuda", lambda *ts: None)
    monkeypatch.setattr(cache_mod, "_NEED", {})
    monkeypatch.setattr(torch.cuda, "stream", lambda stream: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0, raising=False)
    stream = None if stream_on is None else types.SimpleNamespace(device=torch.device("cuda", stream_on), cuda_stream=5)
    cache, i32 = host_cache(), torch.int32
    kv = torch.zeros((2, 3, 4, 64), dtype=torch.bfloat16)
    table, lens = torch.zeros((2, 2), dtype=i32), torch.zeros(2, dtype=i32)
    z, t, f = torch.zeros((2, 9)), torch.zeros(2, dtype=i32), torch.zeros(2)
    calls = [lambda s: cs.cache_append(cache, kv, kv, table, lens, stream=s),
             lambda s: cs.cache_evict(cache, table, lens, torch.zeros((2, 4, 32)), 4, table.clone(), stream=s),
             lambda s: cs.token_logprobs(z, t, stream=s),
             lambda s: cs.token_logprobs_backward(z, t, f, f, f, stream=s)]
    if stream is None:                          # (the attention enters the given stream, and its device with it)
        calls.append(lambda s: cs.cache_attention(kv, cache, table, lens, stream=s))
    for call in calls:
        with pytest.raises(ValueError, match="device|stream"):
            call(stream)
    assert not fake.calls
    if current != -1:
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: -1)
        for call in calls:
            call(None)
        assert len(fake.calls) == 5


@pytest.mark.parametrize("ws", [torch.zeros(1 << 20, dtype=torch.uint8, device="meta"),
                                torch.zeros(1 << 20, dtype=torch.uint8)[::2],
                                torch.zeros(1, dtype=torch.uint8).expand(1 << 20), [0]],
                         ids=["another device", "not contiguous", "one byte of memory", "no tensor"])
def test_a_workspace_that_the_kernels_cannot_write_is_refused(lib, ws):
    with pytest.raises((ValueError, TypeError)):
        attend(host_cache(), 2, 4, 8, ws=ws)
    assert not lib.calls


@pytest.mark.parametrize("dtype", [torch.uint8, torch.int8, torch.float32])
def test_a_workspace_of_any_type_is_used(lib, dtype):
    ws = torch.zeros(1 << 16, dtype=dtype)
    attend(host_cache(), 2, 4, 8, ws=ws)
    assert lib.workspaces() == [(ws.data_ptr(), 1 << 16)]


@pytest.fixture
def host_scores(monkeypatch):
    """score_tokens over CPU tensors, by torch's own operations without a graph."""
    def forward(logits, targets, top=0, suppress_ids=()):
        lse = torch.logsumexp(logits.detach(), -1)
        lp = logits.detach().gather(1, targets.long()[:, None])[:, 0] - lse
        return lp, torch.zeros_like(lse), lse, None, None

    def backward(logits, targets, lse, ent, g_lp, *_, **__):
        hot = torch.nn.functional.one_hot(targets.long(), logits.shape[1])
        return g_lp[:, None] * (hot - torch.softmax(logits.detach(), -1))

    monkeypatch.setattr(score_mod, "token_logprobs", forward)
    monkeypatch.setattr(score_mod, "token_logprobs_backward", backward)
    return torch.randn((3, 7), generator=torch.Generator().manual_seed(2), requires_grad=True)


@pytest.mark.parametrize("loss", [lambda lp: lp.sum(), lambda lp: (lp ** 2).sum()])
def test_the_gradient_of_a_gradient_is_refused(host_scores, loss):
    """A penalty on the gradient, alone or beside the loss itself, is not dropped in silence."""
    z, t = host_scores, torch.tensor([1, 0, 6], dtype=torch.int32)
    lp = cs.score_tokens(z, t)[0]
    g, = torch.autograd.grad(loss(lp), z, create_graph=True)
    want, = torch.autograd.grad(loss(torch.log_softmax(z, 1)[[0, 1, 2], t.long()]), z)
    assert torch.allclose(g, want, atol=1e-6)
    with pytest.raises(RuntimeError, match="differentiated again"):
        (loss(lp) + (g ** 2).sum()).backward()
    lp = cs.score_tokens(z, t)[0]
    z.grad = None
    loss(lp).backward()
    assert torch.allclose(z.grad, want, atol=1e-6) and not z.grad.requires_grad


def test_evict_refuses_weights_that_overlap_the_moved_ones():
    """2 rows of 4 heads of 256 tokens: 8192 bytes."""
    for off in (-8188, -4096, -4, 0, 4, 4096, 8188):
        assert evict(fake_cache(), lo=FAKE + (1 << 16), wo=FAKE + off) == INVALID, off


@pytest.mark.parametrize("kw", [dict(suppress_ids=(3, (1 << 32) + 5)), dict(suppress_ids=(-(1 << 32),)),
                                dict(top=(1 << 32) + 2), dict(top=-(1 << 32))])
def test_numbers_that_do_not_fit_are_refused(monkeypatch, kw):
    """They would reach the library as others: 2^32 + 5 as id 5."""
    fake = FakeLib()
    monkeypatch.setattr(score_mod, "_lib", fake)
    monkeypatch.setattr(score_mod, "_need_cuda", lambda *ts: None)
    monkeypatch.setattr(score_mod, "_raw_stream", lambda stream, index: STREAM)
    monkeypatch.setattr(score_mod, "_empty", lambda shape, dtype, device, stream: torch.empty(0, dtype=dtype))
    z, t, f = torch.zeros((2, 9)), torch.zeros(2, dtype=torch.int32), torch.zeros(2)
    with pytest.raises(ValueError):
        cs.token_logprobs(z, t, **kw)
    if "suppress_ids" in kw:
        with pytest.raises(ValueError):
            cs.token_logprobs_backward(z, t, f, f, f, out=torch.zeros_like(z), **kw)
    assert not fake.calls


@pytest.mark.parametrize("call", [score, grad])
def test_a_top_far_past_the_most_is_unsupported(call):
    for top in (33, 1 << 29, (1 << 30) - 1, (1 << 31) - 1):
        assert call(V=1 << 30, stride=1 << 30, top=top) == UNSUPPORTED, top


def test_attention_refuses_an_output_over_the_queries():
    """2 x 4 queries of 8 heads of 128: 16384 bytes, contiguous at strides 4096, 1024, 128."""
    whole = I3(4096, 1024, 128)
    for off in (-16384 + 16, -16, 16, 2048, 16384 - 16):
        assert c_attend(fake_cache(), s=whole, out=FAKE + off) == INVALID, off
    assert c_attend(fake_cache(), s=whole, w=FAKE + (1 << 16)) == INVALID           # (the weights read q again)
    packed = I3(4 * 1536, 1536, 128)
    for off in (0, 16, 2 * (4 * 1536 + 3 * 1536 + 1024) - 16, -16384 + 16):
        assert c_attend(fake_cache(), s=packed, out=FAKE + off) == INVALID, off
