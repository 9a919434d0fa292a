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


# ---------------------------------------------------------------- outputs on another stream
MS = 2_000_000        # about a millisecond of torch.cuda._sleep


def _outputs_of_every_call(qs):
    """name -> a call with a default output on `stream`; all inputs ready beforehand."""
    new, old, h_q, h_kv, plen = [40, 300, 7], [3, 0, 200], 8, 2, 500
    q, kc, vc, cu, lens = _case(2, new, old, h_q, h_kv)
    pk, pv = _prefix(3, h_kv, plen)
    plen_d = _i32([plen])
    g = _gen(4)
    qkv = _randn(g, sum(new), (h_q + 2 * h_kv) * D, dtype=torch.float32)
    ka, va = torch.zeros_like(kc), torch.zeros_like(vc)
    w = _randn(g, 512, 1024, dtype=torch.float32)
    wq, ws = qs.quantize_weights(w)
    x = _randn(g, 16, 1024)
    freq = 10000.0 ** (-torch.arange(64, dtype=torch.float64, device="cuda") / 64)
    table = qs.rope_table(freq, 600)
    size = {op: qs.workspace_size(op, 16, 512, 1024, 128) for op in (qs.OP_GEMM_W4A4, qs.OP_GEMM_W4A16)}
    work = torch.zeros(max(size.values()), dtype=torch.uint8, device="cuda")
    dec = torch.zeros(qs.attn_workspace_size(3, 1, h_q, h_kv, 300), dtype=torch.uint8, device="cuda")
    return {
        "qkv_rope_append": lambda s: qs.qkv_rope_append(qkv, lens, 0, ka, va, h_q, table, cu=cu, stream=s),
        "attn_prefill": lambda s: qs.attn_prefill(q, cu, lens, kc, vc, h_q, stream=s),
        "attn_prefix": lambda s: qs.attn_prefix(q, lens, 0, kc, vc, h_q, pk, pv, plen_d, cu=cu, stream=s),
        "rope_table": lambda s: qs.rope_table(freq, 600, stream=s),
        "attn_decode": lambda s: qs.attn_decode(qkv[:3], lens, 0, kc, vc, h_q, 300, work=dec, stream=s),
        "gemm_w4a4": lambda s: qs.gemm_w4a4(x, wq, ws, work=work, stream=s),
        "gemm_w4a16": lambda s: qs.gemm_w4a16(x, wq, ws, work=work, stream=s),
        "cast_bf16": lambda s: qs.cast_bf16(w, stream=s),
    }


CALLS = ["qkv_rope_append", "attn_prefill", "attn_prefix", "rope_table", "attn_decode", "gemm_w4a4", "gemm_w4a16",
         "cast_bf16"]


@pytest.mark.parametrize("name", CALLS)
def test_default_output_is_memory_of_the_named_stream(qs, name):
    """What the current stream still has queued on memory that it freed does not reach an output of another
    stream; and what it reads of the output is not given away while it reads."""
    call = _outputs_of_every_call(qs)[name]
    want = call(None)
    side = torch.cuda.Stream()
    call(side)                                              # (its code is loaded)
    torch.cuda.synchronize()
    late = [torch.empty_like(want) for _ in range(3)]
    torch.cuda._sleep(20 * MS)
    for t in late:
        t.fill_(7)                                          # runs after the sleep ...
    del t, late                                             # ... in memory that is free from here on
    out = call(side)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    torch.cuda._sleep(20 * MS)
    got = out.clone()                                       # read after the sleep
    del out
    with torch.cuda.stream(side):
        fresh = [torch.full_like(want, 9) for _ in range(3)]
    torch.cuda.synchronize()
    assert torch.equal(got, want) and len(fresh) == 3
