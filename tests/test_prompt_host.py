"""Host-side checks of the prompt path that need no GPU: argument checks before any launch, the binding's
checks of its tensors, and how the attention's work is shared out."""
import ctypes
import os
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = ctypes.c_void_p(0x10000)      # 16-byte aligned, never dereferenced: validation fails first
FAR = ctypes.c_void_p(0x10000000000)
ODD = ctypes.c_void_p(0x10004)       # 4-byte aligned only


@pytest.fixture(scope="module")
def lib():
    from quantized_speculative_decoding_packed_b200 import build
    build.build()
    from quantized_speculative_decoding_packed_b200 import qspec
    return qspec


def test_every_entry_point_is_bound(lib):
    for name in ("qspec_rope_table", "qspec_qkv_rope_append", "qspec_attn_prefill", "qspec_attn_prefix",
                 "qspec_attn_prefill_workspace_size", "qspec_attn_prefix_workspace_size"):
        assert name in lib.EXPORTED and hasattr(lib.LIB, name)


def _rope(lib, **kw):
    a = dict(qkv=FAKE, ld=1024, n=6, b=2, cu=None, hq=4, hkv=2, d=128, qg=None, kg=None, eps=1e-6, table=FAKE,
             positions=10, rot=128, plen=None, lens=FAKE, off=0, kc=FAKE, vc=FAKE, lmax=8, q=FAR, ldq=512, flags=0,
             ws=None, nb=0)
    a.update(kw)
    return lib.LIB.qspec_qkv_rope_append(a["qkv"], a["ld"], a["n"], a["b"], a["cu"], a["hq"], a["hkv"], a["d"], a["qg"],
                                         a["kg"], a["eps"], a["table"], a["positions"], a["rot"], a["plen"], a["lens"],
                                         a["off"], a["kc"], a["vc"], a["lmax"], a["q"], a["ldq"], a["flags"], a["ws"],
                                         a["nb"], None)


@pytest.mark.parametrize("kw", [
    dict(qkv=None), dict(lens=None), dict(kc=None), dict(vc=None), dict(q=None),
    dict(d=64), dict(hq=5), dict(hkv=0), dict(b=0), dict(b=65536), dict(n=0), dict(n=7), dict(lmax=0), dict(off=-1),
    dict(ld=1020), dict(ld=1026), dict(ldq=504), dict(ldq=516), dict(flags=2, ldq=514), dict(flags=4),
    dict(rot=12), dict(rot=136), dict(rot=-8), dict(table=None), dict(positions=0),
    dict(eps=-1.0), dict(eps=float("nan")),
    dict(qkv=ODD), dict(q=ODD), dict(kc=ODD), dict(vc=ODD), dict(table=ODD), dict(qg=ODD), dict(kg=ODD),
    dict(cu=ctypes.c_void_p(0x10002)), dict(plen=ctypes.c_void_p(0x10002)),
    dict(q=FAKE), dict(q=FAKE, flags=2, ldq=512),       # over the projection, with rows of another length
    dict(q=ctypes.c_void_p(0x10000 + 512), flags=2, ldq=1024),
    dict(ws=FAKE, nb=128), dict(ws=ODD, nb=256),
])
def test_rope_append_rejects(lib, kw):
    assert _rope(lib, **kw) == 1


@pytest.mark.parametrize("args", [
    (None, 64, 8, FAKE, None), (FAKE, 64, 8, None, None), (FAKE, 0, 8, FAKE, None), (FAKE, 12, 8, FAKE, None),
    (FAKE, 136, 8, FAKE, None), (FAKE, 64, 0, FAKE, None), (ctypes.c_void_p(0x10004), 64, 8, FAKE, None),
    (FAKE, 64, 8, ODD, None),
])
def test_rope_table_rejects(lib, args):
    assert lib.LIB.qspec_rope_table(*args) == 1


def _prefill(lib, **kw):
    a = dict(q=FAKE, ldq=512, n=6, b=2, cu=FAKE, hq=4, hkv=2, d=128, lens=FAKE, kc=FAKE, vc=FAKE, lmax=8, out=FAR,
             ldo=512, ws=FAKE, nb=1 << 40)
    a.update(kw)
    return lib.LIB.qspec_attn_prefill(a["q"], a["ldq"], a["n"], a["b"], a["cu"], a["hq"], a["hkv"], a["d"], a["lens"],
                                      a["kc"], a["vc"], a["lmax"], a["out"], a["ldo"], a["ws"], a["nb"], None)


def _prefix(lib, **kw):
    a = dict(q=FAKE, ldq=512, n=6, b=2, cu=None, hq=4, hkv=2, d=128, lens=FAKE, off=0, kc=FAKE, vc=FAKE, lmax=8,
             pk=FAKE, pv=FAKE, pmax=16, plen=FAKE, out=FAR, ldo=512, ws=FAKE, nb=1 << 40)
    a.update(kw)
    return lib.LIB.qspec_attn_prefix(a["q"], a["ldq"], a["n"], a["b"], a["cu"], a["hq"], a["hkv"], a["d"], a["lens"],
                                     a["off"], a["kc"], a["vc"], a["lmax"], a["pk"], a["pv"], a["pmax"], a["plen"],
                                     a["out"], a["ldo"], a["ws"], a["nb"], None)


SHARED = [
    dict(q=None), dict(lens=None), dict(kc=None), dict(vc=None), dict(out=None), dict(ws=None),
    dict(d=64), dict(hq=5), dict(hq=0), dict(hkv=0), dict(hq=129, hkv=1, ldq=129 * 128, ldo=129 * 128),
    dict(b=0), dict(b=65536), dict(n=0), dict(lmax=0),
    dict(ldq=504), dict(ldq=516), dict(ldo=504), dict(ldo=516),
    dict(q=ODD), dict(kc=ODD), dict(vc=ODD), dict(out=ODD), dict(ws=ODD), dict(lens=ctypes.c_void_p(0x10002)),
    dict(out=FAKE), dict(out=ctypes.c_void_p(0x10000 + 5 * 1024)),       # over the queries
]


@pytest.mark.parametrize("kw", SHARED + [dict(cu=None), dict(cu=ctypes.c_void_p(0x10002))])
def test_prefill_rejects(lib, kw):
    assert _prefill(lib, **kw) == 1


@pytest.mark.parametrize("kw", SHARED + [dict(n=7), dict(off=-1), dict(pk=None), dict(pv=None), dict(plen=None),
                                         dict(pmax=0), dict(pk=ODD), dict(pv=ODD), dict(plen=ctypes.c_void_p(0x10002))])
def test_prefix_rejects(lib, kw):
    assert _prefix(lib, **kw) == 1


def test_call_with_packed_arguments_rejects(lib):
    """qspec_call: the number of arguments, integers that do not fit, and what the calls themselves refuse."""
    q = lib._PREFILL_ARGS
    good = [0x10000, 512, 6, 2, 0x10000, 4, 2, 128, 0x10000, 0x10000, 0x10000, 8, 0x10000000000, 512, 0x10000, 1 << 40]
    call = lambda op, args, n, fmt=q: lib.LIB.qspec_call(op, fmt.pack(*args), n, None)      # noqa: E731
    assert lib.LIB.qspec_call(1, None, 16, None) == 1
    for op, n in ((0, 16), (1, 15), (1, 21), (2, 16), (3, 16), (-1, 16)):
        assert call(op, good, n) == 1
    for at, value in ((3, 1 << 31), (3, 0), (5, 1 << 32), (7, 64), (11, -(1 << 40)), (13, 500), (15, -1), (0, 0)):
        bad = list(good)
        bad[at] = value
        assert call(1, bad, 16) == 1
    rope = [0x10000, 1024, 6, 2, 0, 4, 2, 128, 0, 0, 1e-6, 0x10000, 10, 128, 0, 0x10000, 0, 0x10000, 0x10000, 8,
            0x10000000000, 512, 0, 0, 0]
    for at, value in ((10, -1.0), (22, 4), (22, 1 << 32), (22, -1), (24, -1), (13, 12), (16, -1)):
        bad = list(rope)
        bad[at] = value
        assert call(0, bad, 25, lib._ROPE_ARGS) == 1


def test_workspace_sizes_refuse_bad_shapes(lib):
    for n, b, h, kv in ((0, 1, 1, 1), (1, 0, 1, 1), (1, 65536, 1, 1), (1, 1, 0, 1), (2 ** 31, 1, 1, 1), (2 ** 30, 1, 64, 8),
                        (1, 1, 4, 0), (1, 1, 4, 3), (1, 1, 129, 1)):
        assert lib.attn_prefix_workspace_size(n, b, h, kv) == 0


def test_binding_checks_its_tensors(lib):
    q = torch.zeros(4, 512, dtype=torch.bfloat16)
    qkv = torch.zeros(4, 1024)
    cache = torch.zeros(2, 2, 16, 128, dtype=torch.bfloat16)
    lens = torch.zeros(2, dtype=torch.int32)
    cu = torch.zeros(3, dtype=torch.int32)
    pre = torch.zeros(2, 16, 128, dtype=torch.bfloat16)
    plen = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        lib.attn_prefill(q, cu, lens, cache, cache, 4)                       # host tensors
    with pytest.raises(ValueError):
        lib.attn_prefix(q.float(), lens, 0, cache, cache, 4, pre, pre, plen)
    with pytest.raises(ValueError):
        lib.qkv_rope_append(qkv, lens, 0, cache, cache, 4, None)
    with pytest.raises(ValueError):
        lib.rope_table(torch.zeros(64), 10)                                  # fp32 frequencies


def test_prompt_schedule(tmp_path):
    from quantized_speculative_decoding_packed_b200 import build as b
    exe = tmp_path / "prompt_schedule_check"
    src = os.path.join(ROOT, "tests", "prompt_schedule_check.cu")
    cmd = [b.nvcc(), "-std=c++17", "-O1", "-gencode", "arch=compute_100a,code=sm_100a", "-I", b.CSRC, "-o", str(exe), src]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    run = subprocess.run([str(exe)], capture_output=True, text=True)
    assert run.returncode == 0 and run.stdout.startswith("ok"), run.stdout
