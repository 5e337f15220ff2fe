"""The norm with rotation where every block takes many steps: rings that are
used again, groups of tokens that change inside a block (at a batch's end too),
blocks shared out between queries and keys, weight gradients summed over steps,
rows copied ahead while results are written in place. Against the fp64 oracle,
tolerances as in test_gpu_norm_rope.py."""
import numpy as np
import pytest
import torch

import exact_attention_134_b200 as attn
from test_gpu_norm_rope import HALF_BF16, _case, _np, _want

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    attn.lib()


CASES = [
    # B, N, Hq, Hkv, d, rot, axes, interleaved, packed, weights: steps of a block (of 296)
    (1, 2003, 40, 8, 128, 128, 1, False, False, torch.float32),   # 10, two groups at most
    (3, 7001, 2, 1, 128, 64, 3, True, False, torch.bfloat16),     # 6 or 7, three groups
    (1, 40037, 2, 1, 64, 64, 1, False, True, torch.float32),      # 6 or 7
    (2, 9011, 3, 1, 96, 48, 2, False, False, torch.float32),      # 7 or 8
    (1, 9001, 2, 2, 256, 256, 1, True, True, torch.float32),      # 7 or 8
    (1, 5003, 7, 1, 128, 128, 1, False, True, None),              # 4 or 5
]


@pytest.mark.parametrize("case", CASES)
def test_forward_backward_and_in_place(case):
    packed, d = case[8], case[4]
    rows = 256 // (4 if d <= 64 else 8 if d <= 128 else 16)
    assert -(-case[0] * case[1] // rows) * (case[2] + case[3]) >= 4 * 296
    q, k, args, kw, sections = _case(*case)
    yq, yk = attn.qk_norm_rope(q, k, *args, **kw)
    for y, x, w in ((yq, q, args[2]), (yk, k, args[3])):
        want, mag = _want(x, w, args[0], args[1], sections, case[7], packed)
        assert (np.abs(_np(y) - want) <= HALF_BF16 * np.abs(want) + 2.0 ** -18 * mag).all()
    g = torch.Generator().manual_seed(3)
    dyq, dyk = (torch.randn(x.shape, generator=g).bfloat16().cuda() for x in (q, k))
    dq, dk, dwq, dwk = attn.qk_norm_rope_bwd(q, k, dyq, dyk, *args, **kw)
    for dx, dw, x, w, dy in ((dq, dwq, q, args[2], dyq), (dk, dwk, k, args[3], dyk)):
        want, mag, want_w, terms = _want(x, w, args[0], args[1], sections, case[7], packed, dy=dy)
        assert (np.abs(_np(dx) - want) <= HALF_BF16 * np.abs(want) + 2.0 ** -16 * mag).all()
        assert (w is None) == (dw is None)
        if w is not None:
            assert (np.abs(_np(dw) - want_w) <= 2.0 ** -18 * terms + 2.0 ** -24 * np.abs(want_w)).all()
    # the gradients in the place of what they are made of: the same bits
    gq, gk = dyq.clone(), dyk.clone()
    r = attn.qk_norm_rope_bwd(q, k, gq, gk, *args, dq=gq, dk=gk, **kw)
    assert torch.equal(gq, dq) and torch.equal(gk, dk)
    assert all((a is None and b is None) or torch.equal(a, b) for a, b in zip(r[2:], (dwq, dwk)))
    # and the results, in the projection itself
    attn.qk_norm_rope(q, k, *args, q_out=q, k_out=k, **kw)
    assert torch.equal(q, yq) and torch.equal(k, yk)
    assert attn.get_status()[0] == 0
