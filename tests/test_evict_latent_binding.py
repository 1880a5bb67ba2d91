"""CPU tests of the bindings of the eviction and of the latent cache (evict.py,
latent.py): what they hand to the C calls and return, with the library's entry
points replaced by recorders."""
import pytest
import torch

import hadamard_rotation_preprocessing_amd as hr
from hadamard_rotation_preprocessing_amd import cache as K
from hadamard_rotation_preprocessing_amd import evict as E
from hadamard_rotation_preprocessing_amd import latent as A
from test_cache_binding import BAD_WORK, SPEC, Calls, state

LATENT = hr.LatentSpec(256, 64, 16, hr.QSpec("int", 4, 128, False, "bf16"))


@pytest.fixture
def calls(monkeypatch):
    for s in (SPEC, LATENT):
        s.layout()   # (by the real library)
        K._resolved(s).work.clear()
    c = Calls()
    for module, name in ((K, "_cache_lib"), (E, "_evict_lib"), (A, "_latent_lib")):
        monkeypatch.setattr(module, name, lambda: c)
    monkeypatch.setattr(K, "_stream", lambda device: 0)
    monkeypatch.setattr(torch.cuda, "device", c.on)
    monkeypatch.setattr(K, "_current", lambda: None)    # the tensors' device is the CPU, without an index
    yield c
    for s in (SPEC, LATENT):
        K._resolved(s).work.clear()


def everything(work=None):
    """Every call once, with the scratch that those with scratch take."""
    s = state()
    w, lse = torch.zeros((1, 2, 48)), torch.zeros((2, 4))
    pool = hr.cache_pool(LATENT, 4, device="cpu")
    c, rope = torch.zeros((2, 256)), torch.zeros((2, 64))
    q, r = torch.zeros((2, 4, 256)), torch.zeros((2, 4, 64))
    pq, pk = torch.zeros((2, 4, 192)), torch.zeros((5, 4, 128))
    cu = torch.zeros(2, dtype=torch.int32)
    return [
        lambda: hr.cache_weights(s.q, s.pool, SPEC, s.table, s.lens, lse, w, work=work),
        lambda: hr.cache_evict(s.pool, SPEC, s.table, s.lens, w, 16, work=work),
        lambda: hr.latent_attention(q, r, pool, LATENT, s.table, s.lens, 0.1, lse=True, work=work),
        lambda: hr.cache_update(pool, LATENT, s.table, s.lens, s.parents, s.parents, work=work),
        lambda: hr.cache_compact(pool, LATENT, s.table, s.lens, work=work),
        lambda: hr.latent_append(pool, LATENT, c, rope, s.table, s.lens),
        lambda: hr.latent_read(pool, LATENT, s.table, s.lens, None, 2),
        lambda: hr.latent_prompt_attention(pq, pk, torch.zeros((5, 64)), pk, cu, cu, lse=True),
    ]


NAMES = ["hr_cache_weights", "hr_cache_evict", "hr_latent_attention", "hr_latent_update", "hr_latent_compact", "hr_latent_append",
         "hr_latent_read", "hr_latent_prompt_attention"]


def test_calls_run_on_the_device_of_their_tensors(calls, monkeypatch):
    """With another device current, every entry point makes its C calls with the
    tensors' device current."""
    monkeypatch.setattr(K, "_current", lambda: 5)
    for f in everything(torch.empty(64, dtype=torch.uint8)):
        f()
    assert [n for n, _, _ in calls.seen] == NAMES
    assert all(device == torch.device("cpu") for _, device, _ in calls.seen), calls.seen
    assert calls.device == "current"


@pytest.mark.parametrize("work", BAD_WORK.values(), ids=BAD_WORK)
def test_scratch_of_the_caller_is_checked(calls, work):
    bad, good = everything(work()), everything(torch.empty(100, dtype=torch.float32))
    for f, g in list(zip(bad, good))[:5]:
        before = len(calls.seen)
        with pytest.raises(ValueError, match="work must be"):
            f()
        assert len(calls.seen) == before
        g()
        assert 400 in calls.seen[-1][2]     # its size is given in bytes, whatever its type


def test_scratch_sizes_are_asked_for_once(calls):
    s = state()
    w, lse = torch.zeros((1, 2, 48)), torch.zeros((2, 4))
    for _ in range(3):
        hr.cache_weights(s.q, s.pool, SPEC, s.table, s.lens, lse, w)
    assert [n for n, _, _ in calls.seen] == ["hr_cache_weights_work"] + ["hr_cache_weights"] * 3
    calls.seen.clear()
    hr.cache_weights(s.q, s.pool, SPEC, s.table, s.lens, lse, w, max_q=1)
    hr.cache_attention(s.q, s.pool, SPEC, s.table, s.lens)      # (sizes of its own)
    assert [n for n, _, _ in calls.seen] == ["hr_cache_weights_work", "hr_cache_weights", "hr_cache_attention_work", "hr_cache_attention"]


def test_what_the_calls_return(calls):
    s = state(tokens=0)
    w = torch.ones((1, 2, 48))
    assert hr.cache_weights(s.q, s.pool, SPEC, s.table, s.lens, torch.zeros((0, 4)), w, cu_q=s.cu) is w
    out = dict(table=torch.zeros((1, 3), dtype=torch.int32), lens=torch.zeros(1, dtype=torch.int32),
               refs=torch.zeros(4, dtype=torch.int32), status=torch.zeros(4, dtype=torch.int32))
    assert hr.cache_evict(s.pool, SPEC, s.table, s.lens, w, 16, out=out, work=torch.empty(64)) is out
    for name, t in out.items():
        with pytest.raises(ValueError, match="out"):
            hr.cache_evict(s.pool, SPEC, s.table, s.lens, w, 16, out={**out, name: t.long()}, work=torch.empty(64))
    two = hr.cache_pool(SPEC, 4, 2, "cpu")
    r = hr.cache_evict(two, SPEC, s.table, s.lens, torch.ones((2, 1, 2, 48)), 16, 1, 2, work=torch.empty(64))
    assert {k: tuple(v.shape) for k, v in r.items()} == dict(table=(1, 3), lens=(1,), refs=(4,), status=(4,))
    assert calls.seen[-1][2][1:3] == (2, 4) and calls.seen[-1][2][9:13] == (48, 16, 1, 2)
    pool = hr.cache_pool(LATENT, 4, device="cpu")
    c, rope = hr.latent_read(pool, LATENT, s.table, s.lens, None, 7, dtype=torch.float32)
    assert c.shape == (7, 256) and rope.shape == (7, 64) and c.dtype is rope.dtype is torch.float32
    q, r = torch.zeros((0, 4, 256)), torch.zeros((0, 4, 64))
    o, lse = hr.latent_attention(q, r, pool, LATENT, s.table, s.lens, 0.1, cu_q=s.cu, lse=True)
    assert o.shape == (0, 4, 256) and lse.shape == (0, 4)
    assert isinstance(hr.latent_attention(q, r, pool, LATENT, s.table, s.lens, 0.1, cu_q=s.cu, lse=False), torch.Tensor)
    pq, pk, cu = torch.zeros((0, 4, 128)).bfloat16(), torch.zeros((0, 4, 64)).bfloat16(), torch.zeros(1, dtype=torch.int32)
    o, lse = hr.latent_prompt_attention(pq, pk, torch.zeros((0, 64)).bfloat16(), pk, cu, cu, lse=True)
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)


def test_scale_that_float32_does_not_hold(calls):
    f = everything(torch.empty(64, dtype=torch.uint8))
    f[0]()
    assert calls.seen[-1][2][11] == 0.0        # (the default)
    with pytest.raises(ValueError, match="scale"):
        s = state()
        hr.cache_weights(s.q, s.pool, SPEC, s.table, s.lens, torch.zeros((2, 4)), torch.zeros((1, 2, 48)), scale=1e-60)
