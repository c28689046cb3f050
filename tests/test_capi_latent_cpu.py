"""CPU checks of the latent cache's C ABI and binding (bad host-side arguments are refused before
any CUDA call), and of the 64-bit forms that the GPU tests compare with."""
import ctypes
import math

import pytest
import torch

from long_context_speculative_gb300 import build as lib_build
from long_context_speculative_gb300 import rapid

import _latent

P = ctypes.c_void_p(256)        # a fake, aligned device address (never dereferenced)
ODD = ctypes.c_void_p(264)      # 8-byte aligned only
BYTE = ctypes.c_void_p(257)
F = ctypes.c_float


@pytest.fixture(scope="module")
def lib():
    lib_build.build()
    return rapid.lib()


def _refused(call, good, changes, status=-1):
    for i, bad in changes:
        args = list(good)
        args[i] = bad
        assert call(*args) == status, (i, bad)


def _strides(call, good, at, count):
    for i in range(count):
        for bad in (4, -8):       # 8 bytes of bf16; negative
            s = [4096] * count
            s[i] = bad
            args = list(good)
            args[at] = (ctypes.c_int64 * count)(*s)
            assert call(*args) == -1, (i, bad)


def test_latent_append(lib):
    # kv kv_strides q q_strides B n H weight eps inv flags prefix row_offset n_rows q_out cache type cap stream
    good = [P, None, P, None, 2, 11, 16, P, F(1e-6), P, 0, P, P, P, P, P, 1, 4096, None]
    _refused(lib.rapid_latent_append, good,
             [(0, None), (2, None), (4, 0), (5, 0), (5, (1 << 30) + 1), (6, 0), (6, 1025), (8, F(-1.0)),
              (8, F(float("nan"))), (8, F(float("inf"))), (9, None), (10, 2), (11, None), (14, None),
              (15, None), (16, 0), (16, 3), (17, 0), (17, (1 << 29) + 1), (0, ODD), (2, ODD), (7, ODD),
              (14, ODD), (15, ODD), (9, BYTE), (11, BYTE), (12, BYTE), (13, BYTE)])
    _strides(lib.rapid_latent_append, good, 1, 2)
    _strides(lib.rapid_latent_append, good, 3, 6)


def test_latent_read(lib):
    # cache type B cap n first n_rows rows stream
    good = [P, 2, 2, 4096, 100, P, P, P, None]
    _refused(lib.rapid_latent_read, good,
             [(0, None), (7, None), (1, 0), (2, 0), (3, 0), (3, (1 << 29) + 1), (4, 0), (4, (1 << 30) + 1),
              (0, ODD), (7, ODD), (5, BYTE), (6, BYTE)])


def test_latent_commit(lib):
    one = (ctypes.c_void_p * 1)(256)
    # caches layers type B cap n_q prefix path n_accepted stream
    good = [one, 1, 1, 2, 4096, 11, P, P, P, None]
    _refused(lib.rapid_latent_commit, good,
             [(0, None), (0, (ctypes.c_void_p * 1)(None)), (0, (ctypes.c_void_p * 1)(264)), (1, 0), (1, 129),
              (2, 0), (3, 0), (4, 0), (4, (1 << 29) + 1), (5, 0), (5, 65), (6, None), (7, None), (8, None),
              (6, BYTE), (7, BYTE), (8, BYTE)])


def test_latent_attn(lib):
    size = lib.rapid_latent_attn_workspace_size
    need = size(1, 128, 11, 4096, 1)
    assert need > 0 and size(1, 1, 1, 1, 2) > 0
    for i, bad in [(0, 0), (0, 65536), (1, 0), (1, 1025), (2, 0), (2, 65), (3, 10), (3, (1 << 29) + 1),
                   (4, 0), (4, 3)]:
        args = [1, 128, 11, 4096, 1]
        args[i] = bad
        assert size(*args) == 0, (i, bad)
    assert size(65535, 1024, 64, 64, 1) == 0                    # queries
    assert size(400, 1, 1, 1 << 29, 1) == 0                     # tiles of rows, counted in 32 bits
    # many sequences take one split each and no room for parts
    assert size(4000, 128, 11, 4096, 1) < 1 << 20
    # Q cache type B H n_q cap prefix mask scale O LSE ws bytes stream
    good = [P, P, 1, 1, 128, 11, 4096, P, None, F(0.0), P, P, P, need, None]
    _refused(lib.rapid_latent_attn, good,
             [(0, None), (1, None), (7, None), (10, None), (11, None), (12, None), (2, 0), (3, 0), (4, 0),
              (5, 0), (5, 65), (6, 10), (0, ODD), (1, ODD), (10, ODD), (12, ODD), (7, BYTE), (11, BYTE),
              (9, F(float("inf"))), (9, F(float("nan")))])
    _refused(lib.rapid_latent_attn, good, [(13, need - 1)], status=-3)


def test_latent_prefill_attn(lib):
    size = lib.rapid_latent_prefill_attn_workspace_size
    need = size(1, 100, 16, 5000)
    assert need > size(1, 8192, 64, 8192) > 0                   # few blocks have room for split keys
    for i, bad in [(0, 0), (0, 65536), (1, 0), (2, 0), (2, 1025), (3, 0), (3, (1 << 29) + 1)]:
        args = [1, 100, 16, 5000]
        args[i] = bad
        assert size(*args) == 0, (i, bad)
    assert size(65535, 1 << 20, 16, 5000) == 0                  # queries
    # Q K V K_rope strides B n H kv_rows prefix n_rows scale O LSE ws bytes stream
    good = [P, P, P, P, None, 1, 100, 16, 5000, P, P, F(0.0), P, P, P, need, None]
    _refused(lib.rapid_latent_prefill_attn, good,
             [(0, None), (1, None), (2, None), (3, None), (9, None), (12, None), (13, None), (14, None),
              (5, 0), (6, 0), (7, 0), (7, 1025), (8, 0), (0, ODD), (1, ODD), (2, ODD), (3, ODD), (12, ODD),
              (14, ODD), (9, BYTE), (10, BYTE), (13, BYTE), (11, F(float("inf"))), (11, F(float("nan")))])
    _refused(lib.rapid_latent_prefill_attn, good, [(15, need - 1)], status=-3)
    _strides(lib.rapid_latent_prefill_attn, good, 4, 11)
    # a row that repeats: heads of K (more than one of them) with stride 0
    args = list(good)
    args[4] = (ctypes.c_int64 * 11)(*[4096] * 5, 0, *[4096] * 5)
    assert lib.rapid_latent_prefill_attn(*args) == -1


def test_binding_refuses_cpu_tensors_and_wrong_shapes(lib):
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype)   # noqa: E731
    cache, one = z(1, 64, 576), z(1, dtype=torch.int32)
    for call in (lambda: rapid.latent_append(z(1, 3, 576), cache, one, z(32, dtype=torch.float32)),
                 lambda: rapid.latent_read(cache, one, 5),
                 lambda: rapid.LatentLayerTable([cache]),
                 lambda: rapid.LatentLayerTable([]),
                 lambda: rapid.latent_attn(z(1, 16, 3, 576), cache, one),
                 lambda: rapid.latent_prefill_attn(z(1, 3, 2, 192), z(1, 9, 2, 128), z(1, 9, 2, 128),
                                                   z(1, 9, 64), one)):
        with pytest.raises(rapid.RapidError):
            call()


def test_reference_scale_and_rows():
    s = _latent.group_scale(torch.tensor([448.0, 448.1, 0.0, 1e-30, 3.0, 7.0 * 2 ** -9], dtype=torch.float64))
    assert s.tolist() == [1.0, 2.0, 1.0, 2.0 ** -64, 2.0 ** -7, 2.0 ** -15]
    cache = _latent.make_cache((2, 3), True, torch.Generator().manual_seed(1))
    assert cache.shape == (2, 3, _latent.Q8_ROW) and _latent.values(cache).abs().max() < 50
    code, rope, scale = _latent.parts(cache)
    assert torch.equal(_latent.pack(code, rope, scale), cache)


def test_reference_attention_by_hand():
    # two rows seen with equal scores, latent vectors of ones and threes
    cache = torch.zeros((1, 4, 576)).bfloat16()
    cache[0, 0, :512], cache[0, 1, :512], cache[0, 2] = 1.0, 3.0, float("nan")
    Q = torch.zeros((1, 1, 1, 576)).bfloat16()
    O, L, _, _ = _latent.attn(Q, cache, torch.tensor([1]))
    assert torch.equal(O, torch.full_like(O, 2.0)) and abs(float(L) - math.log(2)) < 1e-15
    O, L, _, _ = _latent.attn(Q, cache, torch.tensor([0]), torch.zeros((1, 1, 1)))
    assert float(O.abs().max()) == 0.0 and float(L) == -math.inf


def test_reference_expansion_agrees_with_absorption():
    g = torch.Generator().manual_seed(2)
    H, n, P = 2, 3, 5
    rows = torch.randn((P + n, 576), generator=g).double()
    up_k, up_v = torch.randn((2, H, 128, 512), generator=g).double() / 20
    q = torch.randn((1, n, H, 192), generator=g).double()
    K = torch.einsum("hdc,jc->jhd", up_k, rows[:, :512])[None]
    V = torch.einsum("hdc,jc->jhd", up_v, rows[:, :512])[None]
    O, L, _, _ = _latent.prefill(q, K, V, rows[None, :, 512:], torch.tensor([P]))
    Q = torch.cat([torch.einsum("bihd,hdc->bhic", q[..., :128], up_k), q[..., 128:].transpose(1, 2)], -1)
    O2, L2, _, _ = _latent.attn(Q, rows[None], torch.tensor([P]))
    assert torch.allclose(torch.einsum("hdc,bhic->bihd", up_v, O2), O, rtol=1e-12, atol=1e-12)
    assert torch.allclose(L, L2, rtol=1e-12)


def test_reference_rotation_by_hand():
    x = torch.zeros((1, 64))
    x[0, 0], x[0, 32] = 3.0, 4.0
    inv = torch.zeros(32)
    inv[0] = 1.0
    y, size = _latent.turn(x, [3], inv, False)
    assert abs(float(y[0, 0]) - (3 * math.cos(3) - 4 * math.sin(3))) < 1e-14
    assert abs(float(y[0, 32]) - (4 * math.cos(3) + 3 * math.sin(3))) < 1e-14 and float(size[0, 32]) == 7.0
