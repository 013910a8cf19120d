"""The C ABI of the grouped products (``include/qgmm_mm.h``, libqgmm_mm.so) on the host:
exports, struct layout, and every check that refuses a call before anything is
launched.  No test here reaches a kernel launch."""
import ctypes as C
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "qgmm_mm.h")
FAKE = 1 << 20   # a pointer that no call below dereferences


@pytest.fixture(scope="module")
def q(qgmm):
    qgmm.mm_lib()
    return qgmm


def test_library_exports_what_the_header_declares(q):
    from quantized_moe_grouped_persistent_b200 import mm
    declared = set(re.findall(r"^qgmm_status\s+(qgmm_\w+)\s*\(", open(HEADER).read(), re.M))
    out = subprocess.run(["nm", "-D", "--defined-only", mm.MM_LIB_PATH], capture_output=True, text=True,
                         check=True).stdout
    assert {s for s in re.findall(r" T (\w+)$", out, re.M) if s.startswith("qgmm")} == declared
    assert declared == set(mm.MM_EXPORTS)


def test_problem_layout_matches_the_header(q, tmp_path):
    names = [n for n, _ in q.QgmmMmProblem._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "qgmm_mm.h"\nint main(void) {\n'
                   'printf("size %zu\\n", sizeof(qgmm_mm_problem));\n'
                   + "".join(f'printf("{n} %zu\\n", offsetof(qgmm_mm_problem, {n}));\n' for n in names)
                   + 'printf("%d %d %d %d\\n", QGMM_T_BF16, QGMM_T_F16, QGMM_T_F32, QGMM_T_MXFP4);\nreturn 0; }\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    lines = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.strip().split("\n")
    got = dict(line.split() for line in lines[:-1])
    assert int(got["size"]) == C.sizeof(q.QgmmMmProblem)
    for n in names:
        assert int(got[n]) == getattr(q.QgmmMmProblem, n).offset, n
    assert lines[-1].split() == [str(v) for v in (q.QGMM_T_BF16, q.QGMM_T_F16, q.QGMM_T_F32, q.QGMM_T_MXFP4)]


def _prob(q, **kw):
    a = dict(m=64, k=64, n=48, e=4)
    a.update(kw)
    return q.make_mm_problem(a.pop("m"), a.pop("k"), a.pop("n"), a.pop("e"), **a)


def _ws(q, p):
    out = C.c_size_t(0)
    return q.mm_lib().qgmm_grouped_mm_workspace(C.byref(p), C.byref(out)), out.value


@pytest.mark.parametrize("kw,code", [
    (dict(m=-1), "SHAPE"), (dict(m=(1 << 24) + 1), "SHAPE"), (dict(k=4), "SHAPE"), (dict(k=0), "SHAPE"),
    (dict(k=100), "SHAPE"), (dict(k=65544), "SHAPE"), (dict(n=0), "SHAPE"), (dict(n=12), "SHAPE"),
    (dict(n=65544), "SHAPE"), (dict(e=0), "SHAPE"), (dict(e=1025), "SHAPE"),
    (dict(ld_x=56), "SHAPE"), (dict(ld_x=68), "SHAPE"), (dict(ld_x=-8), "SHAPE"), (dict(ld_x=(1 << 32) + 8), "SHAPE"),
    (dict(ld_w=40), "SHAPE"), (dict(ld_w=52), "SHAPE"), (dict(ld_w=48, transpose_w=True), "SHAPE"),
    (dict(ld_w=(1 << 22) + 8), "SHAPE"), (dict(ld_y=40), "SHAPE"), (dict(ld_y=50), "SHAPE"), (dict(ld_y=-48), "SHAPE"),
    (dict(x_type=2), "DTYPE"), (dict(x_type=4), "DTYPE"), (dict(x_type=-1), "DTYPE"), (dict(out_type=1), "DTYPE"),
    (dict(out_type=3), "DTYPE"), (dict(x_type=1, out_type=0), "DTYPE"), (dict(group_list_type=2), "DTYPE"),
    (dict(x_type=3, out_type=3, transpose_w=True), "DTYPE"), (dict(x_type=3), "UNSUPPORTED"),
    (dict(x_type=3, transpose_w=True, k=72), "SHAPE"), (dict(x_type=3, transpose_w=True, ld_x=72), "SHAPE"),
    (dict(x_type=3, transpose_w=True, ld_w=72), "SHAPE"),
])
def test_problem_is_refused(q, kw, code):
    assert _ws(q, _prob(q, **kw))[0] == getattr(q, "QGMM_ERR_" + code)
    with pytest.raises(q.QgmmError) as err:
        q.grouped_mm_workspace(_prob(q, **kw))
    assert err.value.code == getattr(q, "QGMM_ERR_" + code)


@pytest.mark.parametrize("kw", [dict(m=0), dict(m=1 << 24), dict(k=8, n=8, e=1), dict(k=65536, n=65536, e=1024),
                                dict(x_type=1, out_type=1), dict(x_type=1, out_type=2), dict(accumulate=True),
                                dict(x_type=3, out_type=0, transpose_w=True), dict(x_type=3, out_type=1, transpose_w=True),
                                dict(x_type=3, out_type=2, transpose_w=True, k=32), dict(ld_x=72, ld_w=56, ld_y=4096)])
def test_problem_is_accepted(q, kw):
    rc, n = _ws(q, _prob(q, **kw))
    assert rc == q.QGMM_OK and n >= 256 and n % 256 == 0


def test_flags_are_checked_in_the_struct_itself(q):
    for name in ("transpose_w", "accumulate"):
        p = _prob(q)
        setattr(p, name, 2)
        assert _ws(q, p)[0] == q.QGMM_ERR_SHAPE


def _calls(q, p, ws_bytes=1 << 30):
    """name -> (function, arguments): x x_scale w w_scale gl y ws | dy w gl dx ws | x dy gl dw ws"""
    L, f = q.mm_lib(), FAKE
    mx = p.x_type == q.QGMM_T_MXFP4
    return {"fwd": (L.qgmm_grouped_mm, [f, f if mx else None, f, f if mx else None, f, f, f, ws_bytes, None]),
            "dgrad": (L.qgmm_grouped_mm_dgrad, [f, f, f, f, f, ws_bytes, None]),
            "wgrad": (L.qgmm_grouped_mm_wgrad, [f, f, f, f, f, ws_bytes, None])}


@pytest.mark.parametrize("call,needed", [("fwd", (0, 2, 4, 5, 6)), ("dgrad", (0, 1, 2, 3, 4)),
                                         ("wgrad", (0, 1, 2, 3, 4))])
def test_null_and_misaligned_pointers(q, call, needed):
    p = _prob(q)
    fn, args = _calls(q, p)[call]
    assert fn(None, *args) == q.QGMM_ERR_NULL_PTR
    group_list = {"fwd": 4}.get(call, 2)
    for i in needed:
        a = list(args)
        a[i] = None
        assert fn(C.byref(p), *a) == q.QGMM_ERR_NULL_PTR, i
        if i != group_list:
            a[i] = FAKE + 8
            assert fn(C.byref(p), *a) == q.QGMM_ERR_ALIGNMENT, i
    a = list(args)
    a[-2] = _ws(q, p)[1] - 1
    assert fn(C.byref(p), *a) == q.QGMM_ERR_WORKSPACE_TOO_SMALL


def test_mxfp4_calls(q):
    p = _prob(q, x_type=3, out_type=2, transpose_w=True)
    calls = _calls(q, p)
    fn, args = calls["fwd"]
    for i in (1, 3):     # the scales
        a = list(args)
        a[i] = None
        assert fn(C.byref(p), *a) == q.QGMM_ERR_NULL_PTR
        a[i] = FAKE + 4
        assert fn(C.byref(p), *a) == q.QGMM_ERR_ALIGNMENT
    for name in ("dgrad", "wgrad"):
        fn, args = calls[name]
        assert fn(C.byref(p), *args) == q.QGMM_ERR_UNSUPPORTED


def test_accumulate_belongs_to_the_weight_gradient(q):
    p = _prob(q, accumulate=True)
    for name in ("fwd", "dgrad"):
        fn, args = _calls(q, p)[name]
        assert fn(C.byref(p), *args) == q.QGMM_ERR_UNSUPPORTED


def test_quantiser_checks(q):
    L, f = q.mm_lib(), FAKE
    quant = lambda x=f, t=0, rows=4, k=64, c=f, s=f: L.qgmm_per_token_quant_mxfp4(x, t, rows, k, c, s, None)
    back = lambda c=f, s=f, rows=4, k=64, o=f, t=0: L.qgmm_mxfp4_dequant(c, s, rows, k, o, t, None)
    for call in (quant, back):
        assert call(t=3) == q.QGMM_ERR_DTYPE and call(t=-1) == q.QGMM_ERR_DTYPE
        for bad in (dict(rows=-1), dict(rows=1 << 31), dict(k=0), dict(k=48), dict(k=65568)):
            assert call(**bad) == q.QGMM_ERR_SHAPE, bad
        assert call(rows=0) == q.QGMM_OK
        assert call(c=None) == q.QGMM_ERR_NULL_PTR and call(s=None) == q.QGMM_ERR_NULL_PTR
        assert call(c=f + 2) == q.QGMM_ERR_ALIGNMENT
    assert quant(x=None) == q.QGMM_ERR_NULL_PTR and quant(x=f + 8) == q.QGMM_ERR_ALIGNMENT
    assert back(o=None) == q.QGMM_ERR_NULL_PTR and back(o=f + 8) == q.QGMM_ERR_ALIGNMENT


def test_binding_refuses_tensors_of_the_host(q):
    import torch
    p = _prob(q)
    x, y = torch.zeros(64, 64, dtype=torch.bfloat16), torch.zeros(64, 48, dtype=torch.bfloat16)
    w, gl = torch.zeros(4, 64, 48, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int64)
    ws = torch.zeros(256, dtype=torch.uint8)
    for call in (lambda: q.grouped_mm(p, x, w, gl, y, ws), lambda: q.grouped_mm_dgrad(p, y, w, gl, x, ws),
                 lambda: q.grouped_mm_wgrad(p, x, y, gl, w, ws),
                 lambda: q.per_token_quant_mxfp4(x, torch.zeros(64, 32, dtype=torch.uint8),
                                                 torch.zeros(64, 2, dtype=torch.uint8)),
                 lambda: q.mxfp4_dequant(torch.zeros(64, 32, dtype=torch.uint8), torch.zeros(64, 2, dtype=torch.uint8), x)):
        with pytest.raises(q.QgmmError) as err:
            call()
        assert err.value.code == q.QGMM_ERR_UNSUPPORTED


def test_workspace_holds_the_parts_of_a_long_sum(q):
    """Few rows and a long sum (forward k, backward n) are summed in parts, in f32 in the workspace,
    which then has to be there; 20 MB hold the parts of any bf16 or fp16 problem."""
    assert _ws(q, _prob(q))[1] == 256
    for kw in (dict(m=1, k=8192, n=1024, e=1), dict(m=1, k=1024, n=8192, e=1), dict(m=3, k=4096, n=264, e=40)):
        p = _prob(q, **kw)
        need = _ws(q, p)[1]
        assert need >= 256 + 2 * 4 * kw["m"] * min(kw["k"], kw["n"]) and need % 256 == 0
        for call in ("fwd", "dgrad", "wgrad"):
            fn, args = _calls(q, p)[call]
            a = list(args)
            a[-2] = need - 1
            assert fn(C.byref(p), *a) == q.QGMM_ERR_WORKSPACE_TOO_SMALL
    big = max(_ws(q, _prob(q, m=m, k=k, n=n, e=e))[1] for m in (1, 2, 17, 64, 65, 100, 256, 257, 1000, 2000, 4700, 9400)
              for k in (8, 200, 256, 1000, 2048, 4096, 9000, 65536) for n in (8, 264, 520, 2048, 9472, 65536)
              for e in (1, 2, 9, 40))
    assert 1 << 20 < big <= 20_000_000


def test_binding_raises_without_library(q, tmp_path, monkeypatch):
    from quantized_moe_grouped_persistent_b200 import mm
    monkeypatch.setattr(mm, "_mm_lib", None)
    monkeypatch.setattr(mm, "MM_LIB_PATH", str(tmp_path / "missing.so"))
    with pytest.raises(ImportError):
        mm.mm_lib()


@pytest.mark.parametrize("t,rows", [(0, 32768), (1, 8192)])
def test_workspace_keeps_the_sums_of_long_16_bit_weight_gradients(q, t, rows):
    """Past the rows of one segment a pair's f32 tile each, for 74 pairs or as many as there are tiles."""
    need = lambda **kw: _ws(q, _prob(q, **{**dict(k=2048, n=1536, e=1, x_type=t, out_type=t), **kw}))[1]
    assert need(m=rows) == 256 and need(m=rows + 1) == 256 + 48 * 262144
    assert need(m=rows + 1, out_type=2) == 256
    assert need(m=1 << 24, n=7168, e=32) == 256 + 74 * 262144 <= 20_000_000
    p = _prob(q, m=rows + 1, k=2048, n=1536, e=1, x_type=t, out_type=t)
    fn, args = _calls(q, p)["wgrad"]
    args[-2] = need(m=rows + 1) - 1
    assert fn(C.byref(p), *args) == q.QGMM_ERR_WORKSPACE_TOO_SMALL


@pytest.fixture
def host(q, monkeypatch):
    """The binding on host tensors, its library's calls recorded instead of made."""
    from quantized_moe_grouped_persistent_b200 import mm

    class Recorder:
        calls = []

        def __getattr__(self, name):
            return lambda *a: self.calls.append(name) or 0

    mm._load_torch()
    monkeypatch.setattr(mm, "_device", lambda: -1)       # what get_device() says of host tensors
    monkeypatch.setattr(mm, "_stream_of", lambda stream, device: 0)
    monkeypatch.setattr(mm, "_mm_lib", Recorder())
    Recorder.calls = []
    return Recorder.calls


@pytest.mark.parametrize("transpose_w", [False, True])
def test_binding_refuses_weights_in_the_other_layout(q, host, transpose_w):
    import torch
    m, k, n, e = 6, 64, 48, 4
    p = q.make_mm_problem(m, k, n, e, transpose_w=transpose_w)
    x, y = torch.zeros(m, k, dtype=torch.bfloat16), torch.zeros(m, n, dtype=torch.bfloat16)
    gl, ws = torch.zeros(e, dtype=torch.int64), torch.zeros(256, dtype=torch.uint8)
    calls = lambda w: (lambda: q.grouped_mm(p, x, w, gl, y, ws), lambda: q.grouped_mm_dgrad(p, y, w, gl, x, ws),
                       lambda: q.grouped_mm_wgrad(p, x, y, gl, w, ws))
    right, wrong = ((e, n, k), (e, k, n)) if transpose_w else ((e, k, n), (e, n, k))
    for call in calls(torch.zeros(wrong, dtype=torch.bfloat16)):
        with pytest.raises(q.QgmmError) as err:
            call()
        assert err.value.code == q.QGMM_ERR_SHAPE
    assert not host
    for shape in (right, (e * right[1], right[2]), (e * k * n,), (e + 1, *right[1:])):
        for call in calls(torch.zeros(shape, dtype=torch.bfloat16)):
            call()
    assert len(host) == 12
    p = q.make_mm_problem(m, k, k, e, transpose_w=transpose_w)     # square: the layouts look alike
    q.grouped_mm(p, x, torch.zeros(e, k, k, dtype=torch.bfloat16), gl, torch.zeros_like(x), ws)


def test_binding_refuses_mxfp4_weights_in_the_other_layout(q, host):
    import torch
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    p = q.make_mm_problem(6, 64, 48, 4, x_type=3, out_type=2, transpose_w=True)
    gl, y = torch.zeros(4, dtype=torch.int64), torch.zeros(6, 48)
    call = lambda w, s: q.grouped_mm(p, u8(6, 32), w, gl, y, u8(256), x_scale=u8(6, 2), w_scale=s)
    call(u8(4, 48, 32), u8(4, 48, 2))
    for w, s in ((u8(4, 32, 48), u8(4, 48, 2)), (u8(4, 48, 32), u8(4, 2, 48))):
        with pytest.raises(q.QgmmError) as err:
            call(w, s)
        assert err.value.code == q.QGMM_ERR_SHAPE
    assert len(host) == 1


def test_binding_refuses_what_is_missing(q, host):
    import torch
    x, w = torch.zeros(6, 64, dtype=torch.bfloat16), torch.zeros(4, 64, 48, dtype=torch.bfloat16)
    y, gl = torch.zeros(6, 48, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int64)
    codes, sf = torch.zeros(6, 32, dtype=torch.uint8), torch.zeros(6, 2, dtype=torch.uint8)
    p = q.make_mm_problem(6, 64, 48, 4)
    for call, code in ((lambda: q.grouped_mm(p, x, w, gl, y, None), "NULL_PTR"),
                       (lambda: q.grouped_mm_dgrad(p, y, w, gl, x, None), "NULL_PTR"),
                       (lambda: q.grouped_mm_wgrad(p, x, y, gl, w, None), "NULL_PTR"),
                       (lambda: q.per_token_quant_mxfp4(None, codes, sf), "NULL_PTR"),
                       (lambda: q.per_token_quant_mxfp4(x, None, sf), "NULL_PTR"),
                       (lambda: q.mxfp4_dequant(codes, None, x), "NULL_PTR"),
                       (lambda: q.mxfp4_dequant(codes, sf, None), "NULL_PTR"),
                       (lambda: q.per_token_quant_mxfp4(FAKE, codes, sf), "SHAPE"),
                       (lambda: q.mxfp4_dequant(codes, sf, FAKE), "SHAPE")):
        with pytest.raises(q.QgmmError) as err:
            call()
        assert err.value.code == getattr(q, "QGMM_ERR_" + code)
    assert not host
    q.per_token_quant_mxfp4(x, FAKE, FAKE)                # pointers go through
    q.mxfp4_dequant(FAKE, FAKE, x)
    q.grouped_mm(p, FAKE, FAKE, FAKE, FAKE, FAKE, ws_bytes=256)
    assert host == ["qgmm_per_token_quant_mxfp4", "qgmm_mxfp4_dequant", "qgmm_grouped_mm"]


@pytest.mark.parametrize("kw", [
    dict(k=4096, n=1024, e=4), dict(k=7168, n=2048, e=32), dict(k=65536, n=8, e=1), dict(k=256, n=256, e=1, x_type=1, out_type=1),
    dict(k=16, n=24, e=30, x_type=1, out_type=1), dict(k=2048, n=520, e=3, out_type=2),
    dict(k=16384, n=264, e=2, x_type=3, transpose_w=True), dict(k=1056, n=360, e=40, x_type=3, out_type=2, transpose_w=True),
    dict(k=2048, n=7168, e=8, x_type=3, transpose_w=True)])
def test_workspace_serves_the_same_problem_with_fewer_rows(q, kw):
    """A call of m rows takes the workspace of M >= m; it is refused on its own need less one, at the latest."""
    def accepts(m, nbytes):
        p = _prob(q, m=m, **kw)
        names = ("fwd",) if p.x_type == 3 else ("fwd", "dgrad", "wgrad")
        for fn, args in (_calls(q, p)[c] for c in names):
            a = list(args)
            a[-2] = nbytes
            a[0] = FAKE + 8                                # refused later, as misaligned: nothing is launched
            rc = fn(C.byref(p), *a)
            if rc == q.QGMM_ERR_WORKSPACE_TOO_SMALL:
                return False
            assert rc == q.QGMM_ERR_ALIGNMENT
        return True

    sizes = sorted({1, 2, 3, 7, 24, 25, 64, 65, 95, 96, 97, 255, 256, 257, 500, 1000, 1600, 2000, 4999, 9472, 20000, 32768,
                    32769, 40000, 70000, 300000, 1 << 24})
    needs = {m: _ws(q, _prob(q, m=m, **kw))[1] for m in sizes}
    assert sorted(needs.values()) == [needs[m] for m in sizes]
    for most in sizes:
        for m in sizes:
            if m <= most:
                assert accepts(m, needs[most]), (m, most)
    assert not any(accepts(m, 255) for m in sizes)
