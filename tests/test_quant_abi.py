"""Argument checks of the calls on caches held in 4 bits: everything that the host can see is
refused before any GPU work (the pointers here are numbers that nothing reads)."""
import ctypes as C
import os
import subprocess

import pytest

from tests.test_paged_cache_abi import BAD_CACHES, ROOT, cache, call, cg  # noqa: F401


def form(cg, **kw):
    vals = dict(channels=256, head_dim=64, bits=4, reserved=0, **{})
    return cg.cg_quant_form(*{**vals, **kw}.values())


def quant_cache(cg, **kw):
    return cache(cg, **{**dict(channels=cg.cg_quant_row(256, 64)), **kw})


def points(cg, c, f):
    L, r, q = cg.lib(), C.byref(c), C.byref(f)
    n = C.c_size_t()
    a = call(cg)
    return {
        "write": lambda l0=0, nl=2, n=1, s=64, k=64, v=64, ts=256, ls=256, kh=None, vh=None, hts=256, hls=0:
            L.cg_quant_write_async(r, q, l0, nl, n, s, k, v, ts, ls, kh, vh, hts, hls, None),
        "read": lambda l0=0, nl=2, n=1, s=64, k=64, v=64, ts=256, ls=256:
            L.cg_quant_read_async(r, q, l0, nl, n, s, k, v, ts, ls, None),
        "workspace": lambda: L.cg_quant_attention_workspace(r, q, C.byref(a), C.byref(n)),
        "attention": lambda ws=4096, nws=1 << 40: L.cg_quant_attention_async(r, q, C.byref(a), ws, nws, None),
    }


BAD_FORMS = [dict(channels=0), dict(channels=65537), dict(channels=-64), dict(head_dim=0), dict(head_dim=12),
             dict(head_dim=48), dict(head_dim=264), dict(bits=8), dict(bits=0), dict(reserved=1)]


@pytest.mark.parametrize("bad", BAD_CACHES + [dict(channels=128), dict(channels=73), dict(k_pool_dev=(1 << 20) + 8),
                                              dict(v_pool_dev=(1 << 20) + 2)], ids=str)
def test_bad_caches_are_refused_by_every_call(cg, bad):
    for name, f in points(cg, quant_cache(cg, **bad), form(cg)).items():
        assert f() == cg.CG_E_INVAL and cg.cg_last_error(), name


@pytest.mark.parametrize("bad", BAD_FORMS, ids=str)
def test_bad_forms_are_refused_by_every_call(cg, bad):
    for name, f in points(cg, quant_cache(cg), form(cg, **bad)).items():
        assert f() == cg.CG_E_INVAL and cg.cg_last_error(), name
    n = C.c_int32(-7)
    assert cg.lib().cg_quant_row(C.byref(form(cg, **bad)), C.byref(n)) == cg.CG_E_INVAL and n.value == -7


def test_row_sizes(cg):
    for channels, d, row in ((1024, 128, 576), (128, 64, 80), (400, 80, 272), (8, 8, 32), (65536, 256, 36864),
                             (65536, 32, 36864), (96, 96, 64)):
        assert 2 * cg.cg_quant_row(channels, d) == row
    with pytest.raises(cg.CgError):
        cg.cg_quant_row(65536, 8)  # 147,456 bytes
    assert cg.lib().cg_quant_row(None, C.byref(C.c_int32())) == cg.CG_E_INVAL
    assert cg.lib().cg_quant_row(C.byref(form(cg)), None) == cg.CG_E_INVAL


def test_null_caches_forms_and_calls(cg):
    L, c, f, a, n = cg.lib(), C.byref(quant_cache(cg)), C.byref(form(cg)), C.byref(call(cg)), C.c_size_t()
    bad = cg.CG_E_INVAL
    assert L.cg_quant_write_async(None, f, 0, 1, 1, 64, 64, 64, 256, 0, None, None, 256, 0, None) == bad
    assert L.cg_quant_write_async(c, None, 0, 1, 1, 64, 64, 64, 256, 0, None, None, 256, 0, None) == bad
    assert L.cg_quant_read_async(None, f, 0, 1, 1, 64, 64, 64, 256, 0, None) == bad
    assert L.cg_quant_read_async(c, None, 0, 1, 1, 64, 64, 64, 256, 0, None) == bad
    for args in ((None, f, a), (c, None, a), (c, f, None)):
        assert L.cg_quant_attention_workspace(*args, C.byref(n)) == bad
        assert L.cg_quant_attention_async(*args, 4096, 1 << 40, None) == bad
    assert L.cg_quant_attention_workspace(c, f, a, None) == bad


def test_numbers_of_write_and_read(cg):
    f = points(cg, quant_cache(cg), form(cg))
    bad, ok = cg.CG_E_INVAL, cg.CG_OK
    for x in ("write", "read"):
        g = f[x]
        assert g(l0=-1) == bad and g(l0=1) == bad and g(nl=-1) == bad and g(l0=2, nl=1) == bad
        assert g(n=-1) == bad and g(n=(1 << 21) + 1) == bad
        assert g(s=None) == bad and g(k=None) == bad and g(v=None) == bad
        assert g(ts=255) == bad and g(ls=-1) == bad and g(ts=1 << 41) == bad and g(ls=1 << 41) == bad
        assert g(nl=0) == ok and g(n=0, s=None, k=None, v=None) == ok
    assert f["write"](kh=64) == bad and f["write"](vh=64) == bad
    assert f["write"](kh=64, vh=64, hts=255) == bad and f["write"](kh=64, vh=64, hls=-1) == bad
    assert f["write"](kh=64, vh=64, n=0) == ok


def test_slots_check_their_numbers(cg):
    L, c = cg.lib(), C.byref(cache(cg))
    go = lambda n=1, r=64, f=64, s=64, t=1, o=64: L.cg_pages_slots_async(c, n, r, f, s, t, o, None)  # noqa: E731
    bad, ok = cg.CG_E_INVAL, cg.CG_OK
    assert go(n=-1) == bad and go(n=9) == bad and go(t=-1) == bad and go(t=(1 << 21) + 1) == bad
    assert go(r=None) == bad and go(s=None) == bad and go(o=None) == bad
    assert go(n=0, r=None, s=None, t=0, o=None) == ok
    assert L.cg_pages_slots_async(None, 1, 64, 64, 64, 1, 64, None) == bad
    assert L.cg_pages_slots_async(C.byref(cache(cg, page_tokens=3)), 1, 64, 64, 64, 1, 64, None) == bad


@pytest.mark.parametrize("bad", [
    dict(layer=-1), dict(layer=2), dict(head_dim=32), dict(head_dim=128), dict(n_heads=0), dict(n_heads=3),
    dict(n_heads=1028), dict(scale=float("nan")), dict(scale=float("inf")), dict(n_seqs=-1), dict(n_seqs=9),
    dict(n_q=-1), dict(n_q=(1 << 20) + 1), dict(n_groups=-1), dict(n_groups=3), dict(max_q=-1), dict(max_prefix=-1),
    dict(max_len=-1), dict(q_stride=248), dict(q_stride=260), dict(out_stride=0), dict(out_stride=1 << 41),
    dict(q_starts_dev=None), dict(group_starts_dev=None), dict(prefix_lens_dev=None), dict(q_dev=None),
    dict(out_dev=None), dict(q_dev=(1 << 12) + 2), dict(out_dev=(1 << 12) + 8)], ids=str)
def test_attention_checks_its_arguments(cg, bad):
    c, a = quant_cache(cg), call(cg, **bad)
    rc = cg.lib().cg_quant_attention_async(C.byref(c), C.byref(form(cg)), C.byref(a), 4096, 1 << 40, None)
    assert rc == cg.CG_E_INVAL and cg.cg_last_error()


def test_attention_checks_memory(cg):
    L, c, f, n = cg.lib(), C.byref(quant_cache(cg)), C.byref(form(cg)), C.c_size_t()
    a = call(cg)
    assert L.cg_quant_attention_workspace(c, f, C.byref(a), C.byref(n)) == cg.CG_OK
    assert n.value >= 16 and n.value % 16 == 0
    go = lambda ws, nws: L.cg_quant_attention_async(c, f, C.byref(a), ws, nws, None)  # noqa: E731
    assert go(None, n.value) == cg.CG_E_INVAL and go(4104, n.value) == cg.CG_E_INVAL
    assert go(4096, n.value - 1) == cg.CG_E_CAPACITY
    for k in (dict(n_seqs=0, n_groups=0), dict(n_q=0)):  # nothing to do touches no pointer
        b = call(cg, q_starts_dev=None, **k)
        assert L.cg_quant_attention_async(c, f, C.byref(b), None, 0, None) == cg.CG_OK


def test_struct_layout_matches_the_header(cg, tmp_path):
    fields = [x for x, _ in cg.cg_quant_form._fields_]
    src = ["#include <stdio.h>", "#include <stddef.h>", '#include "cachegen.h"', "int main(void){",
           'printf("%zu", sizeof(cg_quant_form));']
    src += [f'printf(" %zu", offsetof(cg_quant_form, {x}));' for x in fields]
    (tmp_path / "l.c").write_text("\n".join(src + ["return 0;}"]))
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(tmp_path / "l.c"), "-o", str(tmp_path / "l")],
                   check=True)
    got = subprocess.run([str(tmp_path / "l")], capture_output=True, text=True, check=True).stdout.split()
    assert [int(x) for x in got] == [C.sizeof(cg.cg_quant_form)] + [getattr(cg.cg_quant_form, x).offset for x in fields]
