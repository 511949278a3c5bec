"""The C ABI of the rotary and windowed-attention operators, without a GPU:
exports, defaults, refusals that need no device, and the headers as plain C."""
import ctypes
import math
import os
import re
import shutil
import subprocess
import sys

import numpy as np
import pytest

from chunk_scheduled_communication_gb300 import rope, syn, window

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("header, module", [("syn_rope.h", rope), ("syn_window.h", window)])
def test_library_exports_its_header(header, module):
    src = open(os.path.join(ROOT, "include", header)).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = set(re.findall(r"\b(syn_[a-z0-9_]+)\s*\(", src))
    lib = ctypes.CDLL(syn.LIB_PATH)
    assert names and not [n for n in names if not hasattr(lib, n)]
    assert names == set(module.SIGS)


def test_defaults():
    c = rope.make_cfg()
    assert (c.d, c.d_rot, c.layout, c.base, c.scaling, c.attn_factor) == (128, 128, 0, 10000.0, 0, 0.0)
    w, d = window.WindowCfg(), window.DecodeCfg()
    assert window.lib().syn_window_cfg_default(ctypes.byref(w)) == syn.OK
    assert window.lib().syn_decode_cfg_default(ctypes.byref(d)) == syn.OK
    assert (w.H_q, w.H_kv, w.d, w.window, w.sinks, w.backward) == (1, 1, 128, 0, 0, 0)
    assert (d.max_seqs, d.d, d.page_size) == (1, 128, 64)


def test_null_arguments_are_rejected():
    r, w = rope.lib(), window.lib()
    assert r.syn_rope_plan_destroy(None) == syn.OK and w.syn_window_plan_destroy(None) == syn.OK
    assert w.syn_decode_plan_destroy(None) == syn.OK
    assert r.syn_rope_cfg_default(None) == syn.ERR_INVALID
    assert r.syn_rope_plan_create(None, None) == syn.ERR_INVALID
    assert r.syn_rope_plan_frequencies(None, None, None) == syn.ERR_INVALID
    assert r.syn_rope_backward(None, None, None, None, 0, 0, None) == syn.ERR_INVALID
    assert r.syn_qk_norm_rope_backward(None, None, None, 1e-6, None, 0, 0, None) == syn.ERR_INVALID
    assert w.syn_window_plan_create(None, None, 0, None, None) == syn.ERR_INVALID
    assert w.syn_window_plan_query(None, None) == syn.ERR_INVALID
    assert w.syn_window_sync_status(None, None) == syn.ERR_INVALID
    assert w.syn_decode_sync_status(None, None) == syn.ERR_INVALID


def create_window(lens, **kw):
    c = window.WindowCfg()
    window.lib().syn_window_cfg_default(ctypes.byref(c))
    for k, v in kw.items():
        setattr(c, k, v)
    h, n = ctypes.c_void_p(), np.asarray(lens, np.int64)
    return window.lib().syn_window_plan_create(ctypes.byref(h), ctypes.byref(c), len(n), n.ctypes.data, n.ctypes.data)


@pytest.mark.parametrize("lens, kw, status", [
    ([-1], {}, syn.ERR_INVALID), ([1 << 29], {}, syn.ERR_UNSUPPORTED), ([1 << 28] * 4, {}, syn.ERR_UNSUPPORTED),
    ([4], dict(dtype=2), syn.ERR_UNSUPPORTED), ([4], dict(dtype=7), syn.ERR_INVALID), ([4], dict(d=80), syn.ERR_UNSUPPORTED),
    ([4], dict(H_q=3, H_kv=2), syn.ERR_INVALID), ([4], dict(H_q=2048), syn.ERR_UNSUPPORTED), ([4], dict(window=-1), syn.ERR_INVALID),
    ([4], dict(sinks=-1), syn.ERR_INVALID), ([4], dict(scale=math.nan), syn.ERR_INVALID), ([4], dict(backward=2), syn.ERR_INVALID)])
def test_refused_window_plans(lens, kw, status):
    assert create_window(lens, **kw) == status
    assert syn.lib().syn_last_error()


def test_headers_compile_as_plain_c(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "use_window.c"
    src.write_text(
        '#include "syn_rope.h"\n#include "syn_window.h"\n'
        "int use(const void *q, void *y, const int64_t *pos, const int64_t *lens, void *stream) {\n"
        "    syn_rope_cfg_t rc;\n    syn_rope_plan_t rp;\n    syn_window_cfg_t wc;\n    syn_window_plan_t wp;\n"
        "    if (syn_rope_cfg_default(&rc) || syn_window_cfg_default(&wc)) return -1;\n"
        "    if (syn_rope_plan_create(&rp, &rc) || syn_window_plan_create(&wp, &wc, 1, lens, lens)) return -1;\n"
        "    syn_rope_rows_t r = {q, 128, 128, y, 128, 128, 1};\n"
        "    syn_window_rows_t w = {y, 128, 128};\n"
        "    syn_qk_norm_rope(rp, &r, 0, 0, 0, 1e-6f, 0, pos, 0, 0, 0, 16, stream);\n"
        "    syn_window_attention(wp, &w, &w, &w, &w, 0, stream);\n"
        "    int st = syn_window_sync_status(wp, stream);\n"
        "    syn_window_plan_destroy(wp);\n    syn_rope_plan_destroy(rp);\n    return st;\n}\n")
    r = subprocess.run([gcc, "-std=c11", "-Wall", "-Werror", "-fsyntax-only", "-I", os.path.join(ROOT, "include"), str(src)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


@pytest.mark.parametrize("lens, kw", [
    ([1 << 28] * 3, dict(H_q=1024, H_kv=1024)), ([1 << 28] * 3, dict(H_q=1024, H_kv=2)), ([1 << 20] * 1000, dict(H_q=128, H_kv=1)),
    ([1 << 28] * 3, dict(H_q=48, H_kv=8, backward=1)), ([1] * (1 << 20), dict(H_q=512, H_kv=512))])
def test_more_tiles_than_a_plan_can_hold(lens, kw):
    """Refused before the lists are built: 2^28 tiles are 16 GB."""
    assert create_window(lens, **kw) == syn.ERR_UNSUPPORTED
    assert b"tiles" in syn.lib().syn_last_error()


def test_a_plan_that_host_memory_cannot_hold():
    """An error of the call, not the end of the process (a child with little memory left)."""
    code = (
        "import ctypes, resource, numpy as np\n"
        "from chunk_scheduled_communication_gb300 import syn, window\n"
        "c = window.WindowCfg()\n"
        "window.lib().syn_window_cfg_default(ctypes.byref(c))\n"
        "c.H_q = c.H_kv = 64\n"
        "c.backward = 1\n"
        "n, h = np.array([1 << 28], np.int64), ctypes.c_void_p()\n"
        "have = int(open('/proc/self/statm').read().split()[0]) * resource.getpagesize()\n"
        "resource.setrlimit(resource.RLIMIT_AS, (have + (64 << 20), resource.RLIM_INFINITY))\n"
        "rc = window.lib().syn_window_plan_create(ctypes.byref(h), ctypes.byref(c), 1, n.ctypes.data, n.ctypes.data)\n"
        "assert rc == syn.ERR_UNSUPPORTED and b'memory' in syn.lib().syn_last_error(), rc\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT)
    assert r.returncode == 0, r.stderr
