"""attn_decode's default workspace: streams, threads, captured graphs, shapes one after another."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

D = 128


@pytest.fixture(scope="module")
def qs():
    from quantized_speculative_decoding_packed_b200 import qspec
    return qspec


@pytest.fixture
def fresh(qs, monkeypatch):
    """No default workspace from before; the buffers that the test's own thread gets."""
    buffers = qs._StreamBuffers()
    monkeypatch.setattr(qs, "_ATTN_WS", buffers)
    return buffers


def _inputs(seed, batch, h, ctx, t=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    qkv = torch.randn(batch * t, 3 * h * D, device="cuda", generator=g)
    k, v = (torch.randn(batch, h, ctx, D, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    lens = torch.randint(0, ctx - t + 1, (batch,), dtype=torch.int32, device="cuda", generator=g)
    return qkv, lens, k, v, h, ctx


def _call(qs, a, **kw):
    qkv, lens, k, v, h, ctx = a
    return qs.attn_decode(qkv, lens, 0, k, v, h, ctx, **kw)


def _own(qs, a):
    """The call on a workspace of its own."""
    qkv, lens, k, _, h, ctx = a
    n = qs.attn_workspace_size(lens.numel(), qkv.shape[0] // lens.numel(), h, h, ctx)
    return _call(qs, a, work=torch.zeros(n, dtype=torch.uint8, device="cuda"))


def test_shapes_one_after_another_share_one_buffer(qs, fresh):
    """More arrival counters after fewer, longer contexts after shorter: always as on a workspace of its own,
    and one buffer is held, that of the largest call."""
    shapes = [(2, 2, 400, 1), (16, 8, 600, 1), (3, 1, 2000, 5), (40, 4, 130, 2), (1, 1, 50, 1), (16, 8, 600, 4),
              (64, 4, 300, 1), (2, 2, 400, 1)]
    sets = [_inputs(i, b, h, ctx, t) for i, (b, h, ctx, t) in enumerate(shapes)]
    want = [_own(qs, a) for a in sets]
    order = list(range(len(sets))) + [6, 0, 5, 1, 4, 3, 2, 6, 4, 6]
    got = [(i, _call(qs, sets[i])) for i in order]
    torch.cuda.synchronize()
    for i, out in got:
        assert torch.equal(out, want[i]), shapes[i]
    held = [buffer.numel() for buffer, _ in fresh.of.values()]
    assert held == [max(qs.attn_workspace_size(b, t, h, h, ctx) for b, h, ctx, t in shapes)]


def test_two_streams_and_a_named_one(qs, fresh):
    sets = [_inputs(20 + i, 24, 8, 900) for i in range(3)]
    want = [_own(qs, a) for a in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = []
    for turn in range(10):
        for i, (a, st) in enumerate(zip(sets, streams)):
            if turn % 2:
                got.append((i, _call(qs, a, stream=st)))
            else:
                with torch.cuda.stream(st):
                    got.append((i, _call(qs, a)))
    with torch.cuda.stream(streams[0]):                     # the default stream, named where another is current
        got.append((1, _call(qs, sets[1], stream=torch.cuda.default_stream())))
    torch.cuda.synchronize()
    for i, out in got:
        assert torch.equal(out, want[i])
    assert len({b.data_ptr() for b, _ in fresh.of.values()}) == 4


def test_threads_have_their_own(qs, fresh):
    """Calls of several threads, each of another shape, interleaved on the default stream."""
    sets = [_inputs(30 + i, 4 + 9 * i, 4, 500 + 100 * i) for i in range(4)]
    want = [_own(qs, a) for a in sets]
    torch.cuda.synchronize()
    got, errors = [[] for _ in sets], []

    def run(i):
        try:
            torch.cuda.set_device(0)
            for _ in range(50):
                got[i].append(_call(qs, sets[i]))
        except Exception as e:                              # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(sets))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for i, outs in enumerate(got):
        assert len(outs) == 50 and all(torch.equal(out, want[i]) for out in outs)


def test_captured_first_then_eager_then_grown(qs, fresh):
    """A shape that is first met under capture: eager calls before the first replay, a larger eager call and
    other users of freed memory after it, and a second graph, leave both graphs and every call right."""
    a, b, big = _inputs(40, 8, 4, 700), _inputs(41, 8, 4, 700), _inputs(42, 30, 8, 1500, 3)
    want_a, want_b, want_big = _own(qs, a), _own(qs, b), _own(qs, big)
    first = _inputs(43, 16, 4, 300)
    assert torch.equal(_call(qs, first), _own(qs, first))
    graphs, outs = [], []
    for x in (a, b):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(_call(qs, x))
        graphs.append(graph)
    assert torch.equal(_call(qs, a), want_a) and torch.equal(_call(qs, b), want_b)
    assert torch.equal(_call(qs, big), want_big)            # outgrows the eager buffer
    fill = [torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda") for _ in range(64)]
    for order in ((1, 0), (0, 1), (1, 1, 0)):
        for i in order:
            outs[i].zero_()
            graphs[i].replay()
            assert torch.equal(outs[i], (want_a, want_b)[i])
    assert torch.equal(_call(qs, a), want_a) and torch.equal(_call(qs, big), want_big)
    torch.cuda.synchronize()
    assert all(bool((f == 255).all()) for f in fill)


def test_status_of_a_stopped_attention_clears_its_word_alone(qs):
    """An attn_decode workspace can be smaller than the GEMMs' tickets, which a GEMM's timeout clears: what an
    attention reports (bit 2 of the word) is read and cleared, and nothing behind the word is written."""
    need = qs.attn_workspace_size(1, 1, 1, 1, 50)
    assert need < 4352
    for word, status in ((4, 5), (6, 5), (2, 6)):
        buffer = torch.full((8192,), 7, dtype=torch.uint8, device="cuda")
        buffer[:4] = torch.tensor([word, 0, 0, 0], dtype=torch.uint8)
        assert qs.workspace_status(buffer[:need]) == status
        assert not buffer[:4].any() and bool((buffer[4:] == 7).all())
        assert qs.workspace_status(buffer[:need]) == 0


def test_status_of_the_default_workspace(qs, fresh):
    """What attn_decode reports without `work` can be read, on the stream and thread of the call."""
    qkv, lens, k, v, h, ctx = a = _inputs(50, 3, 2, 300)
    want = _own(qs, a)
    bad = (qkv, lens - 400, k, v, h, ctx)
    assert qs.workspace_status(qs.attn_workspace()) == 0
    _call(qs, bad)
    assert qs.workspace_status(qs.attn_workspace("cuda")) == 6 and qs.workspace_status(qs.attn_workspace()) == 0
    assert torch.equal(_call(qs, a), want)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    _call(qs, bad, stream=side)
    side.synchronize()
    assert qs.workspace_status(qs.attn_workspace()) == 0
    assert qs.workspace_status(qs.attn_workspace(stream=side), stream=side) == 6
    assert torch.equal(_call(qs, a), want) and qs.workspace_status(qs.attn_workspace(k.device)) == 0
