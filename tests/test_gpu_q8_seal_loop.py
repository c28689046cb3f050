"""What a decode loop seals, bit for bit (GPU; calls the C ABI through the binding): the caches
as they stand after commit and advance, sealed by the 64-bit form, against what the library leaves
in pages (K and V), scales, tails and lengths.  And a query that is not a number.
"""
import numpy as np
import pytest
import torch

from long_context_speculative_gb300 import rapid

import _q8
import test_gpu_q8_steps as steps

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _float64(t):
    return t.float().cpu().double().numpy()


@pytest.mark.parametrize("tree", [False, True])
def test_every_step_seals_what_the_tail_holds(tree):
    g = torch.Generator().manual_seed(14 + tree)
    loop = steps.Loop()
    steps._prefill(loop, g)
    Q, O, L = steps._buffers()
    sealed = 0
    for k, s in enumerate(steps._steps(g, 10, tree)):
        steps._attend(loop, s, Q, O, L)
        res = rapid.accept(s["z"], s["q"], s["tok"], s["par"], seed=k)
        loop.kv.commit(loop.tail, res["path"], res["n_accepted"])
        rapid.rapid_kv_advance(loop.tail, res["n_accepted"], steps.NQ, steps.CAP)
        torch.cuda.synchronize()
        K, V, pages, scales, sealed0, tail0 = (t.cpu() for t in loop.state())
        pages = pages.view(torch.float8_e4m3fn)
        loop.seal()
        torch.cuda.synchronize()
        table = loop.table.cpu().numpy()
        for layer in range(steps.LAYERS):
            k64, v64, p64, s64 = (_float64(t[layer]) for t in (K, V, pages, scales))
            sealed2, tail2, bad = _q8.seal(k64, v64, p64, s64, table, sealed0.numpy(), tail0.numpy(), steps.KEEP)
            assert not bad
            assert np.array_equal(_float64(loop.K[layer]), k64) and np.array_equal(_float64(loop.V[layer]), v64)
            assert np.array_equal(_float64(loop.pages[layer]), p64)
            assert np.array_equal(_float64(loop.scales[layer]), s64)
        assert np.array_equal(loop.sealed.cpu().numpy(), sealed2) and np.array_equal(loop.tail.cpu().numpy(), tail2)
        sealed += int((sealed2 - sealed0.numpy()).sum()) // 64
    assert sealed >= 2                                     # one block of each sequence at least
    assert rapid.rapid_device_error(True) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_query_that_is_not_a_number(dtype):
    # its scores are none, so neither are its sum and its LSE; no other row notices
    c = _q8.cache(1, 1, 128, dtype, [3], [20], 4, seed=26)
    Q = torch.randn((1, 4, 4, 128), generator=torch.Generator().manual_seed(27)).to(dtype)
    at = [c[k] for k in ("page_table", "sealed_len", "tail_len")]
    ref = _q8.attn(Q, c["K"], c["V"], c["pages"], c["scales"], *at)
    Q[0, 2, 1, 5] = float("nan")
    ref[0][0, 2, 1] = float("nan")
    ref[1][0, 2, 1] = float("nan")
    d = {k: v.to(DEV) for k, v in c.items()}
    O, L = rapid.verify_attn_q8(Q.to(DEV), d["K"], d["V"], d["pages"], d["scales"], d["page_table"],
                                d["sealed_len"], d["tail_len"])
    torch.cuda.synchronize()
    _q8.check(O, ref[0], ref[2], "O")
    _q8.check(L, ref[1], ref[3], "LSE")
    assert rapid.rapid_device_error(True) == 0
