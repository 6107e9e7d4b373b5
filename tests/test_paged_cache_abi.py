"""Argument checks of the paged-cache calls: everything that the host can see is
refused before any GPU work (the pointers here are numbers that nothing reads)."""
import ctypes as C
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def cg():
    import kv_cache_compression_anchor_amd as pkg
    if not os.path.exists(pkg.LIB_PATH):
        from kv_cache_compression_anchor_amd import build
        build.build()
    pkg.lib()
    return pkg


def cache(cg, **kw):
    c = cg.cg_paged_cache()
    vals = dict(device=0, layers=2, channels=128, page_tokens=16, num_pages=100, n_rows=8, max_blocks=20,
                reserved=0, k_pool_dev=1 << 20, v_pool_dev=1 << 21, tables_dev=64, lens_dev=64, refs_dev=64,
                status_dev=64)
    for k, v in {**vals, **kw}.items():
        setattr(c, k, v)
    return c


def call(cg, **kw):
    a = cg.cg_attention()
    vals = dict(layer=1, n_heads=4, head_dim=64, scale=0.125, n_seqs=2, n_q=2, n_groups=1, max_q=1,
                max_prefix=64, max_len=100, rows_dev=None, q_starts_dev=64, group_starts_dev=64,
                prefix_lens_dev=64, q_dev=1 << 12, out_dev=1 << 13, lse_dev=None, q_stride=256,
                out_stride=256)
    for k, v in {**vals, **kw}.items():
        setattr(a, k, v)
    return a


BAD_CACHES = [dict(device=-1), dict(layers=0), dict(layers=5000), dict(channels=0), dict(channels=65537),
              dict(page_tokens=0), dict(page_tokens=12), dict(page_tokens=1 << 17),
              dict(page_tokens=65536, channels=32768), dict(num_pages=0), dict(num_pages=(1 << 24) + 1),
              dict(n_rows=0), dict(n_rows=65537), dict(max_blocks=0), dict(max_blocks=1 << 30),
              dict(reserved=1), dict(k_pool_dev=None), dict(v_pool_dev=None), dict(tables_dev=None),
              dict(lens_dev=None), dict(refs_dev=None), dict(status_dev=None)]


def entry_points(cg, c):
    L, r = cg.lib(), C.byref(c)
    n = C.c_size_t()
    return {
        "workspace": lambda: L.cg_pages_workspace(r, C.byref(n)),
        "copy": lambda n=1, a=64, b=64: L.cg_pages_copy_async(r, n, a, b, None),
        "reserve": lambda n=1, a=64, b=64, t=1, ws=4096, nws=1 << 20: L.cg_pages_reserve_async(
            r, n, a, b, t, 64, ws, nws, None),
        "write": lambda l0=0, nl=2, n=1, s=64, k=64, v=64, ts=128, ls=128: L.cg_pages_write_async(
            r, l0, nl, n, s, k, v, ts, ls, None),
        "fork": lambda n=1, a=64, b=64, ws=4096, nws=1 << 20: L.cg_pages_fork_async(
            r, n, a, b, ws, nws, None),
        "free": lambda n=1, a=64: L.cg_pages_free_async(r, n, a, None),
        "compact": lambda ws=4096, nws=1 << 20: L.cg_pages_compact_async(r, None, ws, nws, None),
    }


@pytest.mark.parametrize("bad", BAD_CACHES, ids=str)
def test_bad_caches_are_refused_by_every_call(cg, bad):
    c = cache(cg, **bad)
    for name, f in entry_points(cg, c).items():
        assert f() == cg.CG_E_INVAL, name
        assert cg.cg_last_error()
    n = C.c_size_t()
    assert cg.lib().cg_attention_workspace(C.byref(c), C.byref(call(cg)), C.byref(n)) == cg.CG_E_INVAL
    assert cg.lib().cg_attention_prefix_async(C.byref(c), C.byref(call(cg)), 4096, 1 << 40,
                                              None) == cg.CG_E_INVAL


def test_null_caches_and_calls(cg):
    L, n = cg.lib(), C.c_size_t()
    assert L.cg_pages_workspace(None, C.byref(n)) == cg.CG_E_INVAL
    assert L.cg_pages_workspace(C.byref(cache(cg)), None) == cg.CG_E_INVAL
    assert L.cg_attention_workspace(C.byref(cache(cg)), None, C.byref(n)) == cg.CG_E_INVAL
    assert L.cg_attention_workspace(C.byref(cache(cg)), C.byref(call(cg)), None) == cg.CG_E_INVAL
    assert L.cg_attention_prefix_async(C.byref(cache(cg)), None, 4096, 1 << 40, None) == cg.CG_E_INVAL


def test_page_calls_check_their_numbers(cg):
    f = entry_points(cg, cache(cg))
    bad, cap, ok = cg.CG_E_INVAL, cg.CG_E_CAPACITY, cg.CG_OK
    assert f["copy"](n=-1) == bad and f["copy"](n=101) == bad
    assert f["copy"](a=None) == bad and f["copy"](b=None) == bad
    assert f["copy"](n=0, a=None, b=None) == ok
    assert f["reserve"](n=-1) == bad and f["reserve"](n=9) == bad and f["reserve"](t=-1) == bad
    assert f["reserve"](t=(1 << 21) + 1) == bad
    assert f["reserve"](a=None) == bad and f["reserve"](b=None) == bad and f["reserve"](ws=None) == bad
    assert f["reserve"](ws=4100) == bad and f["reserve"](nws=64) == cap
    assert f["reserve"](n=0, a=None, b=None, t=0) == ok
    assert f["write"](l0=-1) == bad and f["write"](l0=1) == bad and f["write"](nl=-1) == bad
    assert f["write"](l0=2, nl=1) == bad and f["write"](n=-1) == bad
    assert f["write"](s=None) == bad and f["write"](k=None) == bad and f["write"](v=None) == bad
    assert f["write"](ts=127) == bad and f["write"](ls=-1) == bad and f["write"](ts=1 << 41) == bad
    assert f["write"](nl=0) == ok and f["write"](n=0, s=None) == ok
    assert f["fork"](n=-1) == bad and f["fork"](n=9) == bad and f["fork"](a=None) == bad
    assert f["fork"](b=None) == bad and f["fork"](ws=None) == bad and f["fork"](nws=64) == cap
    assert f["fork"](n=0) == ok
    assert f["free"](n=-1) == bad and f["free"](n=9) == bad and f["free"](a=None) == bad
    assert f["free"](n=0, a=None) == ok
    assert f["compact"](ws=None) == bad and f["compact"](ws=8) == bad and f["compact"](nws=64) == cap


@pytest.mark.parametrize("bad", [
    dict(layer=-1), dict(layer=2), dict(head_dim=0), dict(head_dim=12), dict(head_dim=48), dict(head_dim=264),
    dict(n_heads=0), dict(n_heads=3), dict(n_heads=1026), dict(scale=float("nan")), dict(scale=float("inf")),
    dict(n_seqs=-1), dict(n_seqs=9), dict(n_q=-1), dict(n_q=(1 << 20) + 1), dict(n_groups=-1),
    dict(n_groups=3), dict(max_q=-1), dict(max_prefix=-1), dict(max_len=-1), dict(q_stride=248),
    dict(q_stride=260), dict(out_stride=0), dict(out_stride=257), dict(q_stride=1 << 41),
    dict(q_starts_dev=None), dict(group_starts_dev=None), dict(prefix_lens_dev=None), dict(q_dev=None),
    dict(out_dev=None), dict(q_dev=(1 << 12) + 2), dict(out_dev=(1 << 12) + 8)], ids=str)
def test_attention_checks_its_arguments(cg, bad):
    c, a = cache(cg), call(cg, **bad)
    rc = cg.lib().cg_attention_prefix_async(C.byref(c), C.byref(a), 4096, 1 << 40, None)
    assert rc == cg.CG_E_INVAL and cg.cg_last_error()


@pytest.mark.parametrize("scale,ok", [(2.0 ** 127, True), (-2.0 ** 127, True), (1.5 * 2.0 ** 127, False),
                                      (-1.0001 * 2.0 ** 127, False), (3.4e38, False)])
def test_attention_takes_scales_up_to_2_127(cg, scale, ok):
    n = C.c_size_t()
    rc = cg.lib().cg_attention_workspace(C.byref(cache(cg)), C.byref(call(cg, scale=scale)), C.byref(n))
    assert rc == (cg.CG_OK if ok else cg.CG_E_INVAL)


def test_attention_checks_memory(cg):
    L, c, n = cg.lib(), cache(cg), C.c_size_t()
    a = call(cg)
    assert L.cg_attention_workspace(C.byref(c), C.byref(a), C.byref(n)) == cg.CG_OK and n.value >= 16
    go = lambda c, ws, nws: L.cg_attention_prefix_async(C.byref(c), C.byref(a), ws, nws, None)  # noqa: E731
    assert go(c, None, n.value) == cg.CG_E_INVAL and go(c, 4104, n.value) == cg.CG_E_INVAL
    assert go(c, 4096, n.value - 1) == cg.CG_E_CAPACITY
    assert go(cache(cg, k_pool_dev=(1 << 20) + 8), 4096, n.value) == cg.CG_E_INVAL
    # nothing to do is no error and touches no pointer
    for k in (dict(n_seqs=0, n_groups=0), dict(n_q=0)):
        b = call(cg, q_starts_dev=None, **k)
        assert L.cg_attention_prefix_async(C.byref(c), C.byref(b), None, 0, None) == cg.CG_OK


def test_struct_layouts_match_the_header(cg, tmp_path):
    src = ["#include <stdio.h>", "#include <stddef.h>", '#include "cachegen.h"', "int main(void){"]
    structs = {"cg_paged_cache": cg.cg_paged_cache, "cg_attention": cg.cg_attention}
    for st, cls in structs.items():
        src.append(f'printf("{st} %zu\\n", sizeof({st}));')
        src += [f'printf("{st}.{f} %zu\\n", offsetof({st}, {f}));' for f, _ in cls._fields_]
    (tmp_path / "l.c").write_text("\n".join(src + ["return 0;}"]))
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(tmp_path / "l.c"), "-o",
                    str(tmp_path / "l")], check=True)
    got = dict(x.split() for x in subprocess.run([str(tmp_path / "l")], capture_output=True, text=True,
                                                  check=True).stdout.splitlines())
    for st, cls in structs.items():
        assert int(got[st]) == C.sizeof(cls)
        for f, _ in cls._fields_:
            assert int(got[f"{st}.{f}"]) == getattr(cls, f).offset, (st, f)
