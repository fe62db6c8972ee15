"""What the cache and scoring calls do on the host around the library: the
workspaces, streams and devices they pass, and the calls they refuse.  CPU only:
a stand-in for the library records what reaches it, CPU tensors stand for device
tensors."""
import contextlib

import pytest
import torch

from test_binding_checks import cs

from commit_step_gb300 import cache as cache_mod

STREAM = 77


class FakeLib:
    """Records the calls; everything succeeds.  Sizes come from the library."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if name.endswith("_workspace_size"):
            return getattr(cs.lib_handle(), name)

        def call(*args):
            self.calls.append((name, args))
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
    monkeypatch.setattr(cache_mod, "_WS_AT", {}, raising=False)
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
