"""CPU tests of the paged cache's binding (cache.py): what it hands to the C
calls and returns, with the library's entry points replaced by recorders."""
import contextlib
import types

import pytest
import torch

import hadamard_rotation_preprocessing_amd as hr
from hadamard_rotation_preprocessing_amd import cache as K

SPEC = hr.CacheSpec(2, 64, 16, hr.QSpec("int", 4, 64, False, "bf16"))


class Calls:
    """Stand-in for the library: notes every call and the device it ran on."""

    def __init__(self):
        self.seen, self.device = [], "current"
        self.real = K._cache_lib()

    def __getattr__(self, name):
        def call(*args):
            self.seen.append((name, self.device, args))
            if name.endswith("_work"):
                args[-1]._obj.value = 64
            return 0
        return call

    @contextlib.contextmanager
    def on(self, device):
        self.device, before = device, self.device
        yield
        self.device = before


@pytest.fixture
def calls(monkeypatch):
    SPEC.layout()   # (by the real library)
    c = Calls()
    K._resolved(SPEC).work.clear()
    monkeypatch.setattr(K, "_cache_lib", lambda: c)
    monkeypatch.setattr(K, "_stream", lambda device: 0)
    monkeypatch.setattr(torch.cuda, "device", c.on)
    # the tensors here are on the CPU, whose device has no index: None is "theirs"
    monkeypatch.setattr(K, "_current", lambda: None)
    yield c
    K._resolved(SPEC).work.clear()


def state(tokens=2, rows=1):
    i32 = dict(dtype=torch.int32)
    return types.SimpleNamespace(pool=hr.cache_pool(SPEC, 4, device="cpu"), table=torch.zeros((rows, 3), **i32),
                                 lens=torch.zeros(rows, **i32), q=torch.zeros((tokens, 4, 64)), k=torch.zeros((tokens, 2, 64)),
                                 cu=torch.zeros(rows + 1, **i32), parents=torch.zeros(rows, **i32))


def test_no_tokens(calls):
    """An empty call returns what a call returns: out, and lse where asked for."""
    s = state(tokens=0)
    out, lse = hr.cache_attention(s.q, s.pool, SPEC, s.table, s.lens, cu_q=s.cu, lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    given = torch.empty((0, 4))
    out, lse = hr.cache_attention(s.q, s.pool, SPEC, s.table, s.lens, cu_q=s.cu, lse=given)
    assert lse is given
    assert isinstance(hr.cache_attention(s.q, s.pool, SPEC, s.table, s.lens, cu_q=s.cu, lse=False), torch.Tensor)
    # (a tensor without elements may have any strides)
    e = torch.zeros((64, 2, 0)).permute(2, 1, 0)
    hr.cache_append(s.pool, SPEC, e, e, s.table, s.lens, cu_q=s.cu)
    hr.cache_attention(e, s.pool, SPEC, s.table, s.lens, cu_q=s.cu)


BAD_WORK = {
    "another device": lambda: torch.empty(1 << 16, dtype=torch.uint8, device="meta"),
    "strided": lambda: torch.empty(1 << 16, dtype=torch.uint8)[::2],
}


@pytest.mark.parametrize("work", BAD_WORK.values(), ids=BAD_WORK)
def test_scratch_of_the_caller_is_checked(calls, work):
    s = state()
    for f in (lambda w: hr.cache_attention(s.q, s.pool, SPEC, s.table, s.lens, work=w),
              lambda w: hr.cache_update(s.pool, SPEC, s.table, s.lens, s.parents, s.parents, work=w),
              lambda w: hr.cache_compact(s.pool, SPEC, s.table, s.lens, work=w)):
        before = len(calls.seen)
        with pytest.raises(ValueError, match="work must be"):
            f(work())
        assert len(calls.seen) == before
        # and its size is given in bytes, whatever its type
        w = torch.empty(100, dtype=torch.float32)
        f(w)
        args = calls.seen[-1][2]
        assert args[-3:-1] == (w.data_ptr(), 400)


def test_calls_run_on_the_device_of_their_tensors(calls, monkeypatch):
    """With another device current, every entry point makes its C calls with
    the tensors' device current: the default stream is address 0 on each."""
    monkeypatch.setattr(K, "_current", lambda: 5)
    s = state()
    here = s.pool.device
    hr.cache_append(s.pool, SPEC, s.k, s.k, s.table, s.lens)
    hr.cache_attention(s.q, s.pool, SPEC, s.table, s.lens, lse=True)
    hr.cache_update(s.pool, SPEC, s.table, s.lens, s.parents, s.parents, work=torch.empty(64, dtype=torch.uint8))
    hr.cache_compact(s.pool, SPEC, s.table, s.lens, work=torch.empty(64, dtype=torch.uint8))
    assert [n for n, _, _ in calls.seen] == ["hr_cache_append", "hr_cache_attention_work", "hr_cache_attention",
                                             "hr_cache_update", "hr_cache_compact"]
    assert all(device == here for _, device, _ in calls.seen), calls.seen
    assert calls.device == "current"


def test_scale_that_float32_does_not_hold(calls):
    """0 means 1 / sqrt(head_dim); a scale that only rounds to 0 does not."""
    s = state()
    with pytest.raises(ValueError, match="scale"):
        hr.cache_attention(s.q, s.pool, SPEC, s.table, s.lens, scale=1e-60)
    for given, want in ((None, 0.0), (0.0, 0.0), (0.25, 0.25), (1e-40, 1e-40)):
        hr.cache_attention(s.q, s.pool, SPEC, s.table, s.lens, scale=given)
        assert calls.seen[-1][2][10] == want
