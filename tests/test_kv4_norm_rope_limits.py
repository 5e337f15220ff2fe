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
