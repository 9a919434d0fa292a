"""The prompt attention's failure path, made to run on purpose without faulting the GPU.

QSPEC_CALL_TEST_STALL gives the barrier of each CTA's first key tile one arrival too many to wait for: the
waits run out after their second, the CTA gives up (abort flag, status word, drained copies and products,
freed tensor memory) and returns, the joining kernel runs on what there is, the status reads
QSPEC_ERR_TIMEOUT, and the next calls on the same workspace are as ever.
"""
import pytest
import torch

from test_gpu_prompt import _case, _i32, _prefix

pytestmark = pytest.mark.gpu

TIMEOUT = 5


@pytest.fixture(scope="module")
def qs():
    from quantized_speculative_decoding_packed_b200 import qspec
    return qspec


def _stalled(qs, monkeypatch, call):
    """The call with the hook's bit in its number."""
    lib = qs.LIB

    class Stalls:
        def __getattr__(self, name):
            if name != "qspec_call":
                return getattr(lib, name)
            return lambda op, args, n, stream: lib.qspec_call(op | qs.CALL_TEST_STALL, args, n, stream)

    with monkeypatch.context() as m:
        m.setattr(qs, "LIB", Stalls())
        return call()


@pytest.mark.parametrize("new,old,h_q,h_kv,plen", [
    ([200], [0], 8, 2, 0),                     # CTAs of their own, a join
    ([300, 1, 2000], [1000, 4000, 0], 4, 2, 0),           # shares, split items
    ([1] * 100, [60] * 100, 4, 2, 0),          # more sequences than a warp looks after
    ([5, 3, 64] * 20, [3, 700, 64] * 20, 8, 2, 900),      # a prefix taken once, a row of pieces each
    ([400, 300], [100, 0], 8, 2, 700),         # ahead
])
def test_stalled_wait_reports_timeout_and_the_workspace_serves_on(qs, monkeypatch, new, old, h_q, h_kv, plen):
    q, kc, vc, cu, lens = _case(1, new, old, h_q, h_kv)
    pk, pv = _prefix(2, h_kv, max(plen, 1))
    size = max(qs.attn_prefill_workspace_size(), qs.attn_prefix_workspace_size(sum(new), len(new), h_q, h_kv))
    work = torch.zeros(size, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)

    def call():
        if plen:
            return qs.attn_prefix(q, lens, 0, kc, vc, h_q, pk, pv, _i32([plen]), cu=cu, out=out, work=work)
        return qs.attn_prefill(q, cu, lens, kc, vc, h_q, out=out, work=work)

    want = call().clone()
    assert qs.workspace_status(work) == 0
    for _ in range(2):
        _stalled(qs, monkeypatch, call)
        assert qs.workspace_status(work) == TIMEOUT and qs.workspace_status(work) == 0
        out.zero_()
        assert torch.equal(call(), want) and qs.workspace_status(work) == 0
