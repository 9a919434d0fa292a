"""The prompt path as programs may call it: one token in place, on other streams, from threads, captured, with
starts that are out of order and values that are not finite."""
import math

import pytest
import torch

from test_gpu_prompt import D, _case, _check, _gen, _i32, _prefix, _randn, _table

pytestmark = pytest.mark.gpu

BAD_INPUT = 6


@pytest.fixture(scope="module")
def qs():
    from quantized_speculative_decoding_packed_b200 import qspec
    return qspec


@pytest.mark.parametrize("more", [0, 4])
def test_one_token_is_turned_in_place(qs, more):
    """A lone sequence drafting: one row of the projection, its queries turned where they lie."""
    g = _gen(1)
    h_q, h_kv, lens = 8, 2, _i32([40])
    qkv = _randn(g, 1, (h_q + 2 * h_kv) * D + more, dtype=torch.float32)
    kc, vc = _randn(g, 1, h_kv, 50, D), _randn(g, 1, h_kv, 50, D)
    ka, va, before, table = kc.clone(), vc.clone(), qkv.clone(), _table(qs, 128, 64)
    rows = qkv[:, :(h_q + 2 * h_kv) * D]
    apart = qs.qkv_rope_append(rows, lens, 0, ka, va, h_q, table,
                               q_out=torch.empty(1, h_q * D, dtype=torch.float32, device="cuda"))
    qs.qkv_rope_append(rows, lens, 0, kc, vc, h_q, table, q_out=qkv[:, :h_q * D])
    torch.cuda.synchronize()
    assert torch.equal(qkv[:, :h_q * D], apart) and torch.equal(qkv[:, h_q * D:], before[:, h_q * D:])
    assert torch.equal(kc, ka) and torch.equal(vc, va)
    out = qs.attn_prefill(apart.to(torch.bfloat16), _i32([0, 1]), lens, kc, vc, h_q)
    _check(out, [1], [40], apart.to(torch.bfloat16), kc, vc, h_q)
