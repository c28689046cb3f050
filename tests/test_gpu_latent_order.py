"""Latent cache calls whose inputs the call just before them wrote, with nothing in between (GPU;
calls the C ABI through the binding).  The kernels are launched before their predecessors have
ended, so what they read has to be read behind their wait."""
import pytest
import torch

from long_context_speculative_gb300 import rapid

import _latent

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def _no_error_bits():
    torch.cuda.synchronize()
    rapid.rapid_device_error(True)
    yield
    torch.cuda.synchronize()
    assert rapid.rapid_device_error(True) == 0


def _rope(cache, q8, K):
    """Keys for the expanded form: the cache's own where they stand (bf16 rows), else any."""
    return K[:, :, 0, :64] if q8 else cache[..., 512:]


def _chain(q8, wait):
    """Each round attends, appends rows that the last round read back and rotates what the attention wrote,
    reads the new rows, commits some of them and attends in the other form.  Everything that it wrote."""
    g = torch.Generator().manual_seed(5)
    B, n, H, cap = 2, 40, 8, 400
    i32 = torch.int32
    cache = _latent.make_cache((B, cap), q8, g).to(DEV)
    table = rapid.LatentLayerTable([cache])
    rows = torch.randn((B, n, 576), generator=g).to(BF16).to(DEV)
    Qp = torch.randn((B, n, H, 192), generator=g).to(BF16).to(DEV)
    K, V = (torch.randn((B, cap, H, 128), generator=g).to(BF16).to(DEV) for _ in range(2))
    inv = (5e5 ** (-torch.arange(0, 64, 2).double() / 64)).float().to(DEV)
    weight = torch.ones(512, dtype=BF16, device=DEV)
    length = torch.tensor([300, 17], dtype=i32, device=DEV)
    path = torch.full((B, n), -1, dtype=i32)
    path[:, :10] = torch.arange(2, 22, 2)
    path, acc = path.to(DEV), torch.tensor([10, 7], dtype=i32, device=DEV)
    Q = torch.randn((B, H, n, 576), generator=g).to(BF16).to(DEV)
    out = [torch.empty((12, *s), dtype=t, device=DEV) for s, t in (
        ((B, n, H, 128), BF16), ((B, H, n), torch.float32), ((B, n, 576), BF16), ((B, H, n, 512), BF16),
        ((B, H, n), torch.float32), ((B, H, n, 576), BF16))]
    torch.cuda.synchronize()

    def done():
        if wait:
            torch.cuda.synchronize()

    for i in range(12):
        O, L, R, Oa, La, Qr = (x[i] for x in out)
        rapid.latent_prefill_attn(Qp, K, V, _rope(cache, q8, K), length, out=O, lse=L)
        done()
        rapid.latent_append(rows, cache, length, inv, q=O[..., 64:], q_out=Q[..., 512:].transpose(1, 2), kv_weight=weight)
        done()
        rapid.latent_read(cache, length, n, out=R)
        done()
        rapid.latent_attn(Q, cache, length, out=Oa, lse=La)
        done()
        table.commit(length, path, acc)
        done()
        rapid.latent_attn(Q, cache, length, out=Oa, lse=La)
        done()
        Qr.copy_(Q)
        rows = R
    torch.cuda.synchronize()
    return [*out, cache]


@pytest.mark.parametrize("q8", [False, True])
def test_calls_that_read_what_the_last_call_wrote(q8):
    want = _chain(q8, True)
    for _ in range(3):
        for x, y in zip(_chain(q8, False), want):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_append_rotates_queries_that_repeat_and_refuses_to_write_them_over_each_other():
    g = torch.Generator().manual_seed(1)
    B, n, H = 2, 3, 5
    cache = torch.zeros((B, 16, 576), dtype=BF16, device=DEV)
    kv = torch.randn((B, n, 576), generator=g).to(BF16).to(DEV)
    inv = (5e5 ** (-torch.arange(0, 64, 2).double() / 64)).float().to(DEV)
    length = torch.zeros(B, dtype=torch.int32, device=DEV)
    one = torch.randn((B, n, 1, 64), generator=g).to(BF16).to(DEV)
    want = rapid.latent_append(kv, cache, length, inv, q=one.expand(-1, -1, H, -1).contiguous())
    # one row for all heads, read for each of them
    assert torch.equal(rapid.latent_append(kv, cache, length, inv, q=one.expand(-1, -1, H, -1)), want)
    for out in (one.clone().expand(-1, -1, H, -1), one[:, :1].expand(-1, n, -1, -1).expand(-1, -1, H, -1),
                want.flatten().as_strided((B, n, H, 64), (n * H * 64, H * 64, 32, 1))):
        with pytest.raises(rapid.RapidError):
            rapid.latent_append(kv, cache, length, inv, q=want, q_out=out)
    # sizes of 1 have no stride
    assert torch.equal(rapid.latent_append(kv, cache, length, inv, q=one, q_out=one.as_strided((B, n, 1, 64), (n * 64, 64, 0, 1))),
                       want[:, :, :1])


@pytest.mark.parametrize("q8", [False, True])
def test_commit_on_caches_side_by_side_in_any_order(q8):
    g = torch.Generator().manual_seed(2)
    caches = _latent.make_cache((5, 2, 16), q8, g).to(DEV)
    want = caches.clone()
    for b, P in enumerate((3, 8)):
        want[:, b, P + 1:P + 3] = caches[:, b, [P + 2, P + 5]]
    path = torch.tensor([[2, 5, -1, -1, -1, -1]] * 2, dtype=torch.int32, device=DEV)
    two = torch.full((2,), 2, dtype=torch.int32, device=DEV)
    table = rapid.LatentLayerTable([caches[i] for i in (3, 0, 4, 1, 2)])
    table.commit(torch.tensor([3, 8], dtype=torch.int32, device=DEV), path, two)
    assert torch.equal(caches.view(torch.uint8), want.view(torch.uint8))
