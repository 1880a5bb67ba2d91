"""Pages behind the first 4 GiB of a pool: eviction and the latent cache there give
what they give in a small pool with the same pages, byte for byte."""
import pytest
import torch

import hadamard_rotation_preprocessing_amd as hr

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible: the gpu-marked tests need an MI355X")
    hr.lib()


def pools(spec, used, spare):
    """A pool of more than 2^32 bytes whose last pages are a small pool's."""
    far = (1 << 32) // spec.page_bytes + 100
    g = torch.Generator(device=DEV).manual_seed(3)
    near = torch.randint(0, 60, (used + spare, spec.page_bytes), generator=g, device=DEV, dtype=torch.uint8)
    big = torch.zeros((far + used + spare, spec.page_bytes), dtype=torch.uint8, device=DEV)
    big[far:] = near
    table = torch.randperm(used, generator=g, device=DEV).to(torch.int32).view(2, -1)
    return near, big, far, table


def test_eviction():
    spec = hr.CacheSpec(8, 128, 64, hr.QSpec("int", 4, 128, False, "bf16"))
    near, big, far, table = pools(spec, 12, 0)
    lens = torch.tensor([330, 100], dtype=torch.int32, device=DEV)
    for new in (1, 20):                      # few rows, and many
        q = torch.randn((2 * new, 32, 128), device=DEV).bfloat16()
        got = []
        for pool, t in ((near, table), (big, table + far)):
            o, lse = hr.cache_attention(q, pool, spec, t, lens, lse=True)
            w = torch.ones((2, 8, 384), device=DEV)
            got.append((o, hr.cache_weights(q, pool, spec, t, lens, lse, w)))
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert (got[0][1] > 0).all()
    w = torch.rand((2, 8, 384), device=DEV)
    w2 = w.clone()
    a = hr.cache_evict(near, spec, table, lens, w, 90, 4, 30)
    b = hr.cache_evict(big, spec, table + far, lens, w2, 90, 4, 30)
    assert torch.equal(w, w2) and torch.equal(near, big[far:]) and int(big[:far].sum()) == 0
    assert torch.equal(torch.where(a["table"] < 0, -1, a["table"] + far), b["table"]) and a["lens"].tolist() == b["lens"].tolist() == [90, 90]
    assert torch.equal(a["refs"], b["refs"][far:]) and int(b["refs"][:far].sum()) == 0


def test_latents():
    spec = hr.LatentSpec(512, 64, 64, hr.QSpec("int", 4, 128, False, "bf16"))
    near, big, far, table = pools(spec, 12, 0)
    lens = torch.tensor([330, 100], dtype=torch.int32, device=DEV)
    c, rope = torch.randn((200, 512), device=DEV).bfloat16(), torch.randn((200, 64), device=DEV).bfloat16()
    q, qr = torch.randn((8, 48, 512), device=DEV).bfloat16(), torch.randn((8, 48, 64), device=DEV).bfloat16()
    got = []
    for pool, t in ((near, table), (big, table + far)):
        hr.latent_append(pool, spec, c, rope, t, lens)
        hr.latent_append(pool, spec, c.new_zeros((100, 512)).normal_(generator=torch.Generator(device=DEV).manual_seed(1)),
                         rope[:100], t, lens - 100 + 50)
        got.append(hr.latent_attention(q, qr, pool, spec, t, lens, 0.05, lse=True) + hr.latent_read(pool, spec, t, lens, None, 200))
    assert torch.equal(near, big[far:]) and int(big[:far].sum()) == 0
    for x, y in zip(*got):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
