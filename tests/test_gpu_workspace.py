"""Default workspaces: calls of different kinds and shapes without `work` leave each other's alone."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_decode_attention_leaves_the_gemms_tickets(monkeypatch):
    """attn_decode, GEMM, attn_decode of another shape, all on default workspaces: every result as on a fresh one."""
    from quantized_speculative_decoding_packed_b200 import qspec as qs
    g = torch.Generator(device="cuda").manual_seed(3)
    w = torch.randn(512, 2048, device="cuda", generator=g) * 0.02
    wq, ws = qs.quantize_weights(w)
    x = torch.randn(16, 2048, device="cuda", generator=g).to(torch.bfloat16)
    size = qs.workspace_size(qs.OP_GEMM_W4A16, 16, 512, 2048, 128)
    want = qs.gemm_w4a16(x, wq, ws, work=torch.zeros(size, dtype=torch.uint8, device="cuda"))

    def decode(batch, h, own):
        gg = torch.Generator(device="cuda").manual_seed(batch)
        qkv = torch.randn(batch, 3 * h * 128, device="cuda", generator=gg)
        k = torch.randn(batch, h, 400, 128, device="cuda", generator=gg).to(torch.bfloat16)
        lens = torch.full((batch,), 390, dtype=torch.int32, device="cuda")
        n = qs.attn_workspace_size(batch, 1, h, h, 400)
        return qs.attn_decode(qkv, lens, 0, k, k, h, 400,
                              work=torch.zeros(n, dtype=torch.uint8, device="cuda") if own else None)

    monkeypatch.setattr(qs, "_WS_CACHE", {})
    fresh = {s: decode(*s, True) for s in ((2, 2), (16, 8), (3, 1))}
    for s in ((2, 2), (16, 8), (3, 1), (16, 8)):
        assert torch.equal(decode(*s, False), fresh[s]), s
        assert torch.equal(qs.gemm_w4a16(x, wq, ws), want), s
