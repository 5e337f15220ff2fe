"""The largest sizes that the norm with rotation and the 4-bit cache take (no
GPU): what is above them is refused before anything touches CUDA."""
import pytest

import exact_attention_134_b200 as attn
from exact_attention_134_b200 import build as attn_build

P = 0x10000  # a fake, 16-byte-aligned "device pointer": never dereferenced on these paths


@pytest.fixture(scope="module")
def lib():
    attn_build.build()
    return attn.lib()


@pytest.mark.parametrize("page,most", [(16, 0x7fff000), (1024, 0x1fffc0)])
def test_tokens_of_a_page_table(lib, page, most):
    """2^31 - 65536 tokens are taken (and the pool's alignment is looked at next), a page more is not."""
    def calls(mp):
        pool = P + 8
        return (lib.attn_kv4_append(P, P, 64, 64, 64, 64, pool, P, P, P, 1, mp, 8, page, 1, 1, 64, None),
                lib.attn_kv4_gather(pool, P, P, P, 1, mp, 8, page, 1, 1, 64, P, P, None),
                lib.attn_fwd_kv4(P, pool, P, P, P, P, P, 1, mp, 8, page, 1, 1, 1, 1, 64, 1, 0.1, P, 1 << 40, None))
    assert calls(most) == (3, 3, 3)
    assert calls(most + 1) == (2, 2, 2)
    assert calls((2 ** 31 - 16) // page) == (2, 2, 2)  # 2^31 - 16 tokens: 32 behind them pass 2^31


def test_tokens_of_a_norm_rope_call(lib):
    """2^31 - 65536 tokens are taken (and the tensors' alignment is looked at next), one more is not."""
    import ctypes

    def calls(n):
        def s(k):
            return (ctypes.c_longlong * (3 * k))(*[64] * (3 * k))
        return (lib.attn_qk_norm_rope(P + 8, P, P, P, s(4), None, None, 0, None, 0, 0, None, None, 0, 0, 0, 1, n, 1, 1,
                                      64, 0.0, None),
                lib.attn_qk_norm_rope_bwd(P + 8, P, P, P, P, P, s(6), None, None, 0, None, None, None, 0, 0, None, None,
                                          0, 0, 0, 1, n, 1, 1, 64, 0.0, None, 0, None))
    assert calls(2 ** 31 - 65536) == (3, 3)
    assert calls(2 ** 31 - 65535) == (2, 2)
    assert calls(2 ** 31 - 17) == (2, 2)  # rounded up to 64 tokens this passes 2^31


def test_results_that_are_one_tensor_or_the_other_ones_source(lib):
    """q_out and k_out (dq and dk) at one address, or one of them where the other one is read from:
    blocks of the two would write over what they read. Refused, as every pair is."""
    import ctypes
    q, k, a, b, c, d, w = (P + 0x1000 * i for i in range(7))

    def fwd(qo, ko):
        s = (ctypes.c_longlong * 12)(*[64] * 12)
        return lib.attn_qk_norm_rope(q, k, qo, ko, s, w, w, 0, None, 0, 0, None, None, 0, 0, 0, 1, 9, 1, 1, 64, 0.0, None)

    def bwd(dq, dk, weight=w):
        s = (ctypes.c_longlong * 18)(*[64] * 18)
        need = lib.attn_qk_norm_rope_bwd_workspace_size(1, 9, 1, 1, 64)
        return lib.attn_qk_norm_rope_bwd(q, k, a, b, dq, dk, s, weight, weight, 0, w, w, None, 0, 0, None, None, 0, 0, 0, 1,
                                         9, 1, 1, 64, 0.0, None, need, None)  # no workspace: 6 is what comes next
    assert fwd(a, a) == fwd(k, b) == fwd(a, q) == fwd(k, q) == 1
    assert bwd(c, c) == bwd(b, d) == bwd(c, a) == bwd(b, a) == 1
    assert bwd(k, d) == bwd(c, q) == 1
    assert bwd(c, d) == bwd(a, b) == bwd(a, d) == bwd(q, k) == 6
    assert lib.attn_kv4_gather(P, P, P, P, 1, 8, 8, 16, 1, 1, 64, a, a, None) == 1
