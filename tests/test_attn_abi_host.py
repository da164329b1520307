"""The C ABI of softmax attention and its pages on the host: every symbol
declared in include/kda_attn.h and include/kda_pages.h is exported, and invalid
arguments are rejected with the documented status codes before anything is
enqueued (no call here reaches a kernel launch)."""
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
    ("kda_attn.h", {"kda_attn_fwd", "kda_attn_bwd", "kda_attn_bwd_workspace_bytes", "kda_kv_append",
                    "kda_attn_paged_fwd", "kda_attn_paged_workspace_bytes"}),
    ("kda_pages.h", {"kda_kv_resize", "kda_kv_fork", "kda_kv_fork_workspace_bytes", "kda_kv_compact",
                     "kda_kv_compact_workspace_bytes"})])
def test_exports_every_declared_symbol(lib, header, names):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    assert set(re.findall(r"\b(kda_[a-z_0-9]+)\s*\(", text)) == names
    for n in names:
        assert hasattr(lib, n), n


# addresses that are never dereferenced
NAMES = "q k v cu o lse go gq gk gv ws kp vp table len refs want ok src dst tab2 refs2 live data data2".split()
ADDR = {n: 0x7F0000000000 + i * 0x1000000000 for i, n in enumerate(NAMES)}


def ptr(n, off=0):
    return (ADDR[n] + off,)


def call(fn, order, defaults, kw):
    a = dict(defaults)
    a.update(kw)
    return fn(*[ctypes.c_void_p(a[n][0]) if isinstance(a[n], tuple) else a[n] for n in order.split()])


def fwd(lib, **kw):
    d = dict(q=ptr("q"), qs=256, k=ptr("k"), ks=128, v=ptr("v"), vs=128, dt=0, cu=None, n=2, T=10, H=4, G=2, D=64, sc=0.1,
             ca=1, o=ptr("o"), lse=ptr("lse"), st=None)
    return call(lib.kda_attn_fwd, "q qs k ks v vs dt cu n T H G D sc ca o lse st", d, kw)


def test_fwd_refusals(lib):
    assert fwd(lib, dt=2) == DTYPE
    assert fwd(lib, D=96) == SHAPE and fwd(lib, G=3) == SHAPE and fwd(lib, H=0) == SHAPE and fwd(lib, G=0) == SHAPE
    assert fwd(lib, n=-1) == SHAPE and fwd(lib, T=-1) == SHAPE
    for n in "qkvo":
        assert fwd(lib, **{n: None}) == NULLP
        assert fwd(lib, **{n: ptr(n, 8)}) == ALIGN
    assert fwd(lib, lse=ptr("lse", 2)) == ALIGN and fwd(lib, cu=ptr("cu", 1)) == ALIGN
    assert fwd(lib, qs=248) == SHAPE and fwd(lib, ks=120) == SHAPE and fwd(lib, vs=132) == ALIGN
    assert fwd(lib, qs=(1 << 20) + 8) == LARGE
    assert fwd(lib, H=65540, G=2, qs=1 << 20) == LARGE
    assert fwd(lib, T=(1 << 30) + 1, H=1, G=1) == LARGE and fwd(lib, n=2 ** 31 - 1, T=1 << 29) == LARGE
    assert fwd(lib, o=ptr("q", 128)) == ALIAS and fwd(lib, lse=ptr("v")) == ALIAS and fwd(lib, lse=ptr("o")) == ALIAS
    assert fwd(lib, n=0) == OK and fwd(lib, T=0, q=None) == OK


def bwd(lib, **kw):
    d = dict(q=ptr("q"), qs=256, k=ptr("k"), ks=128, v=ptr("v"), vs=128, dt=0, cu=None, n=2, T=10, H=4, G=2, D=64, sc=0.1,
             ca=1, o=ptr("o"), lse=ptr("lse"), go=ptr("go"), gq=ptr("gq"), gqs=256, gk=ptr("gk"), gks=128, gv=ptr("gv"),
             gvs=128, ws=ptr("ws"), wb=1 << 20, st=None)
    return call(lib.kda_attn_bwd, "q qs k ks v vs dt cu n T H G D sc ca o lse go gq gqs gk gks gv gvs ws wb st", d, kw)


def test_bwd_refusals(lib):
    assert bwd(lib, dt=-1) == DTYPE and bwd(lib, D=32) == SHAPE
    for n in "q k v o lse go gq gk gv".split():
        assert bwd(lib, **{n: None}) == NULLP, n
    for n in "q k v o go gq gk gv ws".split():
        assert bwd(lib, **{n: ptr(n, 4)}) == ALIGN, n
    assert bwd(lib, gqs=128) == SHAPE and bwd(lib, gvs=1 << 21) == LARGE and bwd(lib, gks=129) == ALIGN
    need = lib.kda_attn_bwd_workspace_bytes(0, 2, 10, 4, 2, 64, 0)
    assert need >= 2 * 10 * 4 * 4
    assert bwd(lib, wb=need - 1) == WS and bwd(lib, ws=None) == WS
    assert bwd(lib, gq=ptr("q")) == ALIAS and bwd(lib, gk=ptr("go", 64)) == ALIAS and bwd(lib, gv=ptr("lse")) == ALIAS
    assert bwd(lib, gv=ptr("gk", 128)) == ALIAS and bwd(lib, ws=ptr("o")) == ALIAS and bwd(lib, ws=ptr("gq")) == ALIAS
    assert bwd(lib, n=0) == OK
    assert lib.kda_attn_bwd_workspace_bytes(0, 2, 10, 4, 3, 64, 0) == 0


def paged(lib, **kw):
    d = dict(q=ptr("q"), qs=256, dt=0, kp=ptr("kp"), vp=ptr("vp"), ps=2 * 16 * 64, np=9, pg=16, tab=ptr("table"), mp=4,
             len=ptr("len"), cu=None, n=2, T=3, H=4, G=2, D=64, sc=0.1, o=ptr("o"), lse=ptr("lse"), ws=ptr("ws"), wb=1 << 30,
             st=None)
    return call(lib.kda_attn_paged_fwd, "q qs dt kp vp ps np pg tab mp len cu n T H G D sc o lse ws wb st", d, kw)


def test_paged_refusals(lib):
    assert paged(lib, dt=3) == DTYPE and paged(lib, D=256) == SHAPE
    for pg in (0, 8, 24, 512, -16):
        assert paged(lib, pg=pg) == SHAPE, pg
    assert paged(lib, np=-1) == SHAPE and paged(lib, mp=-1) == SHAPE and paged(lib, ps=2047) == SHAPE
    assert paged(lib, ps=2052) == ALIGN and paged(lib, mp=1 << 27) == LARGE and paged(lib, ps=1 << 41) == LARGE
    assert paged(lib, q=None) == NULLP and paged(lib, kp=None) == NULLP and paged(lib, tab=None) == NULLP
    assert paged(lib, len=None) == NULLP and paged(lib, o=None) == NULLP
    assert paged(lib, kp=ptr("kp", 8)) == ALIGN and paged(lib, tab=ptr("table", 2)) == ALIGN
    assert paged(lib, o=ptr("kp", 4096)) == ALIAS and paged(lib, lse=ptr("len")) == ALIAS and paged(lib, o=ptr("q")) == ALIAS
    need = lib.kda_attn_paged_workspace_bytes(0, 2, 3, 4, 2, 64, 16, 1000, 0)
    assert need > 0
    assert paged(lib, mp=1000, wb=need - 1) == WS and paged(lib, mp=1000, ws=None) == WS
    assert paged(lib, mp=1000, ws=ptr("vp")) == ALIAS
    assert paged(lib, n=0) == OK and paged(lib, T=0) == OK
    assert lib.kda_attn_paged_workspace_bytes(0, 2, 3, 4, 2, 64, 17, 1000, 0) == 0


@pytest.mark.parametrize("scale", [float("nan"), float("inf"), -float("inf")])
def test_a_scale_that_is_no_number_is_refused(lib, scale):
    for f in (fwd, bwd, paged):
        assert f(lib, sc=scale) == SHAPE


def test_a_scale_whose_base_2_form_overflows_is_refused(lib):
    for f in (fwd, bwd, paged):
        assert f(lib, sc=3e38) == SHAPE and f(lib, sc=-2.4e38) == SHAPE
        assert f(lib, sc=2.3e38, T=0) == OK and f(lib, sc=-2.3e38, T=0) == OK and f(lib, sc=1e-45, T=0) == OK


def append(lib, **kw):
    d = dict(k=ptr("k"), ks=128, v=ptr("v"), vs=128, dt=0, kp=ptr("kp"), vp=ptr("vp"), ps=2 * 16 * 64, np=9, pg=16,
             tab=ptr("table"), mp=4, len=ptr("len"), cu=None, n=2, T=3, G=2, D=64, st=None)
    return call(lib.kda_kv_append, "k ks v vs dt kp vp ps np pg tab mp len cu n T G D st", d, kw)


def test_append_refusals(lib):
    assert append(lib, dt=5) == DTYPE and append(lib, pg=20) == SHAPE and append(lib, G=0) == SHAPE
    assert append(lib, k=None) == NULLP and append(lib, vp=None) == NULLP and append(lib, len=None) == NULLP
    assert append(lib, ks=64) == SHAPE and append(lib, vs=130) == ALIGN and append(lib, v=ptr("v", 2)) == ALIGN
    assert append(lib, kp=ptr("k")) == ALIAS and append(lib, vp=ptr("kp", 64)) == ALIAS and append(lib, tab=ptr("vp")) == ALIAS
    # pages of one pool side by side are apart: only the missing k is left to say
    assert append(lib, vp=ptr("kp", 4096), ps=4096, k=None) == NULLP
    assert append(lib, T=0) == OK and append(lib, n=0) == OK and append(lib, np=0, kp=None, vp=None) == OK


def resize(lib, **kw):
    d = dict(tab=ptr("table"), len=ptr("len"), refs=ptr("refs"), want=ptr("want"), ok=ptr("ok"), ns=4, mp=4, np=9, pg=16,
             st=None)
    return call(lib.kda_kv_resize, "tab len refs want ok ns mp np pg st", d, kw)


def test_resize_refusals(lib):
    assert resize(lib, pg=48) == SHAPE and resize(lib, ns=-1) == SHAPE and resize(lib, mp=-1) == SHAPE and resize(lib, np=-1) == SHAPE
    assert resize(lib, ns=65537) == LARGE and resize(lib, ns=65536, mp=1 << 15) == LARGE and resize(lib, np=1 << 30) == LARGE
    for n in ("len", "refs", "want"):
        assert resize(lib, **{n: None}) == NULLP, n
    assert resize(lib, tab=None) == NULLP and resize(lib, refs=ptr("refs", 2)) == ALIGN
    assert resize(lib, want=ptr("len")) == ALIAS and resize(lib, ok=ptr("want", 4)) == ALIAS and resize(lib, refs=ptr("table", 16)) == ALIAS
    assert resize(lib, ns=0) == OK


def data(*t):
    n = max(1, len(t))
    return ((ctypes.c_void_p * n)(*[x[0] for x in t]), (ctypes.c_int64 * n)(*[x[1] for x in t]),
            (ctypes.c_int64 * n)(*[x[2] for x in t]), len(t))


GOOD = ((ADDR["data"], 64, 128), (ADDR["data"] + 64, 64, 128))


def fork(lib, t=GOOD, **kw):
    p, b, s, n = data(*t)
    d = dict(tab=ptr("table"), len=ptr("len"), refs=ptr("refs"), src=ptr("src"), dst=ptr("dst"), ok=ptr("ok"), n=3, ns=4, mp=4,
             np=9, pg=16, p=p, b=b, s=s, nt=n, ws=ptr("ws"), wb=1 << 20, st=None)
    return call(lib.kda_kv_fork, "tab len refs src dst ok n ns mp np pg p b s nt ws wb st", d, kw)


def compact(lib, t=GOOD, **kw):
    p, b, s, n = data(*t)
    d = dict(tab=ptr("table"), len=ptr("len"), refs=ptr("refs"), tab2=ptr("tab2"), refs2=ptr("refs2"), live=ptr("live"), ns=4,
             mp=4, np=9, pg=16, p=p, b=b, s=s, nt=n, ws=ptr("ws"), wb=1 << 20, st=None)
    return call(lib.kda_kv_compact, "tab len refs tab2 refs2 live ns mp np pg p b s nt ws wb st", d, kw)


def test_fork_and_compact_refusals(lib):
    D = ADDR["data"]
    for f in (fork, compact):
        assert f(lib, pg=15) == SHAPE and f(lib, ns=-2) == SHAPE and f(lib, nt=-1) == SHAPE and f(lib, nt=17) == LARGE
        assert f(lib, len=None) == NULLP and f(lib, refs=None) == NULLP and f(lib, p=None) == NULLP
        assert f(lib, ((D, 0, 64),)) == SHAPE and f(lib, ((D, 64, 48),)) == SHAPE
        assert f(lib, ((D, 24, 32),)) == ALIGN and f(lib, ((D + 8, 32, 32),)) == ALIGN and f(lib, ((D, 32, 40),)) == ALIGN
        assert f(lib, ((None, 32, 32),)) == NULLP and f(lib, ((D, 1 << 37, 1 << 37),)) == LARGE
        assert f(lib, ((D, 64, 128), (D + 48, 64, 128))) == ALIAS
        assert f(lib, wb=8) == WS and f(lib, ws=None) == WS
        assert f(lib, ((ADDR["table"], 64, 64),)) == ALIAS and f(lib, ((ADDR["ws"], 64, 64),)) == ALIAS
    assert fork(lib, n=-1) == SHAPE and fork(lib, n=65537) == LARGE and fork(lib, n=65536, mp=1 << 17, ns=1) == LARGE
    assert fork(lib, src=None) == NULLP and fork(lib, dst=ptr("dst", 1)) == ALIGN
    assert fork(lib, dst=ptr("len")) == ALIAS and fork(lib, ok=ptr("src")) == ALIAS and fork(lib, n=0) == OK
    assert fork(lib, ((ADDR["src"], 64, 64),)) == ALIAS
    assert compact(lib, tab2=None) == NULLP and compact(lib, refs2=None) == NULLP and compact(lib, live=None) == NULLP
    assert compact(lib, tab2=ptr("table", 4)) == ALIAS and compact(lib, refs2=ptr("table")) == ALIAS
    assert compact(lib, live=ptr("refs")) == ALIAS and compact(lib, tab2=ptr("len")) == ALIAS
    assert lib.kda_kv_compact_workspace_bytes(-1) == 0 and lib.kda_kv_fork_workspace_bytes(-1, 1, 1) == 0
