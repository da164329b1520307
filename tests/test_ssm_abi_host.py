"""The C ABI of the state space scan, its convolution and the draft
verification on the host: every symbol declared in include/kda_ssm.h and
include/kda_spec.h is exported, and invalid arguments are rejected with the
documented status codes before anything is enqueued (no call here reaches a
kernel launch)."""
import ctypes
import os
import re

import pytest

import gated_delta_rule_amd as kda

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULLP, SHAPE, DTYPE, ALIGN, ALIAS, WS, LARGE, HIPERR = range(9)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(kda.library_path()):
        from gated_delta_rule_amd import build
        build.build()
    return kda.load_library()


@pytest.mark.parametrize("header,names", [
    ("kda_ssm.h", {"kda_ssm_conv_fwd", "kda_ssm_conv_step", "kda_ssm_conv_bwd", "kda_ssm_conv_bwd_workspace_bytes",
                   "kda_ssm_chunk_fwd", "kda_ssm_chunk_fwd_workspace_bytes", "kda_ssm_chunk_bwd",
                   "kda_ssm_chunk_bwd_workspace_bytes", "kda_ssm_recurrent_fwd"}),
    ("kda_spec.h", {"kda_verify_drafts", "kda_verify_drafts_workspace_bytes"})])
def test_exports_every_declared_symbol(lib, header, names):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    assert set(re.findall(r"\b(kda_[a-z_0-9]+)\s*\(", text)) == names
    for n in names:
        assert hasattr(lib, n), n


# addresses that are never dereferenced
BASE = 0x7F0000000000
ADDR = {n: BASE + i * 0x1000000000 for i, n in enumerate(
    ["x", "B", "C", "dt", "bias", "A", "D", "S0", "cu", "y", "ST", "ws", "w", "cache", "rx", "nr", "gy", "gx", "gw",
     "gb", "gc", "gS", "gB", "gC", "gdt", "gA", "gD", "gS0", "rB", "rdt", "p", "q", "drafts", "nd", "u", "un", "na",
     "tok"])}


def call(fn, order, defaults, kw):
    a = dict(defaults)
    a.update(kw)
    out = []
    for n in order:
        v = a[n]
        out.append(v if isinstance(v, int) or v is None else ctypes.c_void_p(v[0]))
    return fn(*out)


def ptr(n, off=0):
    return (ADDR[n] + off,)


def conv(lib, **kw):
    d = dict(x=ptr("x"), xs=64, dt=0, w=ptr("w"), bias=ptr("bias"), cache=ptr("cache"), cu=None, n=2, T=10, c=64, W=4,
             act=1, y=ptr("y"), st=None)
    return call(lib.kda_ssm_conv_fwd, "x xs dt w bias cache cu n T c W act y st".split(), d, kw)


def test_conv_fwd_refusals(lib):
    assert conv(lib, dt=2) == DTYPE
    assert conv(lib, c=60) == SHAPE and conv(lib, c=0) == SHAPE
    assert conv(lib, W=1) == SHAPE and conv(lib, W=5) == SHAPE
    assert conv(lib, n=-1) == SHAPE and conv(lib, T=-1) == SHAPE
    assert conv(lib, x=None) == NULLP and conv(lib, w=None) == NULLP and conv(lib, y=None) == NULLP
    assert conv(lib, xs=56) == SHAPE                       # rows closer than their width
    assert conv(lib, xs=68) == ALIGN                       # rows not on 16 bytes
    assert conv(lib, xs=(1 << 23) + 8) == LARGE
    assert conv(lib, x=ptr("x", 8)) == ALIGN and conv(lib, cache=ptr("cache", 4)) == ALIGN
    assert conv(lib, y=ptr("x", 128)) == ALIAS and conv(lib, y=ptr("cache")) == ALIAS
    assert conv(lib, cache=ptr("w")) == ALIAS
    assert conv(lib, n=2 ** 31 - 1, T=2 ** 40) == LARGE
    assert conv(lib, n=0) == OK


def step(lib, **kw):
    d = dict(x=ptr("x"), xs=64, dt=0, w=ptr("w"), bias=None, cache=ptr("cache"), rx=ptr("rx"), rs=64, nr=ptr("nr"),
             B=2, T=4, Tr=4, c=64, W=4, act=1, commit=1, y=ptr("y"), st=None)
    return call(lib.kda_ssm_conv_step, "x xs dt w bias cache rx rs nr B T Tr c W act commit y st".split(), d, kw)


def test_conv_step_refusals(lib):
    assert step(lib, T=65) == SHAPE and step(lib, Tr=65) == SHAPE and step(lib, Tr=-1) == SHAPE
    assert step(lib, cache=None) == NULLP and step(lib, rx=None) == NULLP and step(lib, w=None) == NULLP
    assert step(lib, rs=72, rx=ptr("rx", 2)) == ALIGN and step(lib, nr=ptr("nr", 2)) == ALIGN
    assert step(lib, cache=ptr("rx")) == ALIAS and step(lib, y=ptr("nr")) == ALIAS
    assert step(lib, B=0) == OK


def conv_bwd(lib, **kw):
    d = dict(x=ptr("x"), xs=64, dt=0, w=ptr("w"), bias=ptr("bias"), cache=ptr("cache"), cu=None, n=2, T=10, c=64, W=4,
             act=1, gy=ptr("gy"), gs=64, gx=ptr("gx"), gw=ptr("gw"), gb=ptr("gb"), gc=ptr("gc"), ws=ptr("ws"),
             wsb=1 << 20, st=None)
    return call(lib.kda_ssm_conv_bwd,
                "x xs dt w bias cache cu n T c W act gy gs gx gw gb gc ws wsb st".split(), d, kw)


def test_conv_bwd_refusals(lib):
    need = lib.kda_ssm_conv_bwd_workspace_bytes(20, 64, 4)
    assert need == 5 * 64 * 4                              # one partial sum of 4 taps and the bias
    assert lib.kda_ssm_conv_bwd_workspace_bytes(20, 60, 4) == 0
    assert conv_bwd(lib, wsb=need - 1) == WS and conv_bwd(lib, ws=None) == WS
    assert conv_bwd(lib, gw=None) == NULLP and conv_bwd(lib, gy=None) == NULLP
    assert conv_bwd(lib, gx=ptr("x")) == ALIAS and conv_bwd(lib, gc=ptr("cache")) == ALIAS
    assert conv_bwd(lib, gw=ptr("gb")) == ALIAS and conv_bwd(lib, ws=ptr("gx")) == ALIAS


def scan(lib, **kw):
    d = dict(x=ptr("x"), xs=512, B=ptr("B"), bs=128, C=ptr("C"), cs=128, dt=0, dts=ptr("dt"), bias=None, soft=1,
             A=ptr("A"), D=None, S0=None, cu=None, n=2, T=100, H=8, G=1, N=128, P=64, y=ptr("y"), ST=ptr("ST"),
             ws=None, wsb=0, st=None)
    return call(lib.kda_ssm_chunk_fwd,
                "x xs B bs C cs dt dts bias soft A D S0 cu n T H G N P y ST ws wsb st".split(), d, kw)


def test_chunk_fwd_refusals(lib):
    assert scan(lib, dt=3) == DTYPE
    for bad in (dict(N=32), dict(P=32), dict(H=0), dict(G=3), dict(G=0), dict(T=-1), dict(n=-2)):
        assert scan(lib, **bad) == SHAPE, bad
    assert scan(lib, H=131072, G=1) == LARGE
    assert scan(lib, x=None) == NULLP and scan(lib, A=None) == NULLP and scan(lib, dts=None) == NULLP
    assert scan(lib, xs=504) == SHAPE and scan(lib, bs=132) == ALIGN and scan(lib, cs=2 ** 23 + 8) == LARGE
    assert scan(lib, ST=ptr("ST", 8)) == ALIGN and scan(lib, dts=ptr("dt", 2)) == ALIGN
    assert scan(lib, y=ptr("x")) == ALIAS and scan(lib, ST=ptr("B")) == ALIAS
    assert scan(lib, S0=ptr("ST", 16)) == ALIAS            # partly in place
    big = dict(T=100000, n=1)
    need = kda.ssm_chunk_fwd_workspace_bytes(1, 100000, 8, 1, 128, 64, False)
    assert need > 0
    assert scan(lib, **big, ws=ptr("ws", 8), wsb=need) == ALIGN
    assert scan(lib, **big, ws=ptr("y"), wsb=need) == ALIAS
    assert scan(lib, n=0) == OK


def test_chunk_fwd_plan():
    ws = kda.ssm_chunk_fwd_workspace_bytes
    assert ws(1, 100, 8, 1, 128, 64, False) == 0           # too short to cut
    assert ws(64, 100000, 64, 1, 128, 64, False) == 0      # thousands of chains as they are
    assert ws(1, 100000, 8, 3, 128, 64, False) == 0        # invalid
    # cut: a state and a decay factor per segment and head, whole chunks per segment
    per = 8 * (128 * 64 + 1) * 4
    for varlen in (False, True):
        need = ws(1, 100000, 8, 1, 128, 64, varlen)
        assert need % per == 0 and 2 <= need // per <= 100000 // 64 + 1
    # packed: sequences may start anywhere in a segment
    assert ws(300, 100000, 8, 8, 128, 64, True) in [0] + [(100000 // (64 * k) + 300) * per for k in range(1, 1600)]


def scan_bwd(lib, **kw):
    d = dict(x=ptr("x"), xs=512, B=ptr("B"), bs=128, C=ptr("C"), cs=128, dt=0, dts=ptr("dt"), bias=ptr("bias"), soft=1,
             A=ptr("A"), D=ptr("D"), S0=ptr("S0"), cu=None, n=2, T=100, H=8, G=1, N=128, P=64, gy=ptr("gy"),
             gS=ptr("gS"), gx=ptr("gx"), gxs=512, gB=ptr("gB"), gBs=128, gC=ptr("gC"), gCs=128, gdt=ptr("gdt"),
             gA=ptr("gA"), gD=ptr("gD"), gb=ptr("gb"), gS0=ptr("gS0"), ws=ptr("ws"), wsb=0, st=None)
    return call(lib.kda_ssm_chunk_bwd, ("x xs B bs C cs dt dts bias soft A D S0 cu n T H G N P gy gS gx gxs gB gBs "
                                        "gC gCs gdt gA gD gb gS0 ws wsb st").split(), d, kw)


def test_chunk_bwd_refusals(lib):
    need = lib.kda_ssm_chunk_bwd_workspace_bytes(0, 2, 100, 8, 1, 128, 64, 0, 1)
    assert need > 2 * 4 * 8 * 128 * 64 * 4                 # two states per chunk and head
    assert lib.kda_ssm_chunk_bwd_workspace_bytes(0, 2, 100, 8, 1, 128, 64, 0, 0) == 0
    assert lib.kda_ssm_chunk_bwd_workspace_bytes(1, 2, 100, 8, 1, 128, 64, 0, 1) > need   # shorter chunks
    assert scan_bwd(lib, wsb=need - 1) == WS and scan_bwd(lib, ws=None, wsb=need) == WS
    ok = dict(wsb=need)
    assert scan_bwd(lib, **ok, gA=None) == NULLP and scan_bwd(lib, **ok, gdt=None) == NULLP
    assert scan_bwd(lib, **ok, gxs=500) == SHAPE and scan_bwd(lib, **ok, gBs=132) == ALIGN
    assert scan_bwd(lib, **ok, gx=ptr("x")) == ALIAS and scan_bwd(lib, **ok, gB=ptr("gC")) == ALIAS
    # one buffer of wider rows for the three: columns that touch are fine, columns that overlap are not
    wide = dict(gxs=768, gBs=768, gCs=768, gx=ptr("gx"), gB=ptr("gx", 1024))
    assert scan_bwd(lib, **ok, **wide, gC=ptr("gx", 1264)) == ALIAS
    assert scan_bwd(lib, **ok, **wide, gC=ptr("gx", 1280), ws=ptr("gx", 2048)) == ALIAS   # reaches the workspace's check
    assert scan_bwd(lib, **ok, gS0=ptr("gS", 16)) == ALIAS


def rec(lib, **kw):
    d = dict(x=ptr("x"), xs=512, B=ptr("B"), bs=128, C=ptr("C"), cs=128, dt=0, dts=ptr("dt"), bias=None, soft=1,
             A=ptr("A"), D=None, rx=ptr("rx"), rxs=512, rB=ptr("rB"), rBs=128, rdt=ptr("rdt"), nr=ptr("nr"),
             S=ptr("S0"), b=2, T=4, Tr=4, H=8, G=1, N=128, P=64, commit=1, y=ptr("y"), st=None)
    return call(lib.kda_ssm_recurrent_fwd,
                "x xs B bs C cs dt dts bias soft A D rx rxs rB rBs rdt nr S b T Tr H G N P commit y st".split(), d, kw)


def test_recurrent_refusals(lib):
    assert rec(lib, T=65) == SHAPE and rec(lib, Tr=65) == SHAPE and rec(lib, N=256) == SHAPE
    assert rec(lib, S=None) == NULLP and rec(lib, rdt=None) == NULLP and rec(lib, C=None) == NULLP
    assert rec(lib, rBs=130) == ALIGN and rec(lib, S=ptr("S0", 4)) == ALIGN
    assert rec(lib, y=ptr("S0")) == ALIAS and rec(lib, S=ptr("rx")) == ALIAS
    assert rec(lib, b=1 << 22) == LARGE                    # more workgroups than a launch takes
    assert rec(lib, b=0) == OK


def verify(lib, **kw):
    d = dict(p=ptr("p"), q=ptr("q"), dt=1, drafts=ptr("drafts"), nd=ptr("nd"), u=ptr("u"), un=ptr("un"), B=2, K=4,
             V=1000, na=ptr("na"), tok=ptr("tok"), ws=ptr("ws"), wsb=32, st=None)
    return call(lib.kda_verify_drafts, "p q dt drafts nd u un B K V na tok ws wsb st".split(), d, kw)


def test_verify_refusals(lib):
    assert lib.kda_verify_drafts_workspace_bytes(2, 4, 1000) == 32
    assert lib.kda_verify_drafts_workspace_bytes(3, 4, 4097) == 3 * 2 * 16
    assert lib.kda_verify_drafts_workspace_bytes(3, 65, 100) == 0
    assert verify(lib, dt=2) == DTYPE and verify(lib, K=65) == SHAPE and verify(lib, V=0) == SHAPE
    assert verify(lib, V=2 ** 31) == LARGE and verify(lib, B=2 ** 24) == LARGE
    assert verify(lib, p=None) == NULLP and verify(lib, u=None) == NULLP and verify(lib, tok=None) == NULLP
    assert verify(lib, p=ptr("p", 8)) == ALIGN and verify(lib, nd=ptr("nd", 1)) == ALIGN
    assert verify(lib, wsb=31) == WS and verify(lib, ws=None) == WS
    assert verify(lib, na=ptr("tok", 4)) == ALIAS and verify(lib, tok=ptr("drafts")) == ALIAS
    assert verify(lib, B=0) == OK


def test_python_refusals_without_a_gpu():
    torch = pytest.importorskip("torch")
    x = torch.zeros(1, 4, 64)
    with pytest.raises(kda.KDAError, match="device tensor"):
        kda.ssm_conv_fwd(x, torch.zeros(64, 4))
    with pytest.raises(kda.KDAError):
        kda.ssm_chunk_fwd(x[..., None], torch.zeros(1, 4, 1), torch.zeros(1), x[..., None], x[..., None])
    with pytest.raises(kda.KDAError):
        kda.verify_drafts(torch.zeros(1, 2, 8), torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, 1), torch.zeros(1))
