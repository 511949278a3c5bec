"""The C ABI of the layer norm, the gated feed-forward block and the gradient
clipping, without a GPU: exports, defaults, refusals that need no device, and the
headers as plain C."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

from chunk_scheduled_communication_gb300 import clip, ffn, norm, syn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("header, module", [("syn_norm.h", norm), ("syn_ffn.h", ffn), ("syn_clip.h", clip)])
def test_library_exports_its_header(header, module):
    src = open(os.path.join(ROOT, "include", header)).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = set(re.findall(r"\b(syn_[a-z0-9_]+)\s*\(", src))
    lib = ctypes.CDLL(syn.LIB_PATH)
    assert names and not [n for n in names if not hasattr(lib, n)]
    assert names == set(module.SIGS)


def test_defaults():
    n, f = norm.NormCfg(), ffn.FfnCfg()
    assert norm.lib().syn_norm_cfg_default(ctypes.byref(n)) == syn.OK
    assert ffn.lib().syn_ffn_cfg_default(ctypes.byref(f)) == syn.OK
    assert (n.dtype, n.d) == (0, 4096)
    assert (f.dtype, f.d, f.d_ff, f.act, f.backward, f.saved_f32, f.timeout_ns) == (0, 4096, 14336, 0, 1, 0, 0)


def test_null_arguments_are_rejected():
    n, f, c = norm.lib(), ffn.lib(), clip.lib()
    assert n.syn_norm_plan_destroy(None) == f.syn_ffn_plan_destroy(None) == c.syn_clip_plan_destroy(None) == syn.OK
    assert n.syn_norm_cfg_default(None) == f.syn_ffn_cfg_default(None) == syn.ERR_INVALID
    assert n.syn_norm_plan_create(None, None) == f.syn_ffn_plan_create(None, None) == syn.ERR_INVALID
    assert c.syn_clip_plan_create(None) == syn.ERR_INVALID
    assert n.syn_layer_norm(None, None, None, None, 1e-5, None, 0, None) == syn.ERR_INVALID
    assert n.syn_layer_norm_backward(None, None, None, None, 1e-5, None, None, None, 0, None) == syn.ERR_INVALID
    assert f.syn_gated_ffn(None, *[None] * 6, 0, None) == syn.ERR_INVALID
    assert f.syn_gated_ffn_backward(None, *[None] * 11, 0, None) == syn.ERR_INVALID
    assert f.syn_ffn_sync_status(None, None) == syn.ERR_INVALID
    assert c.syn_grad_norm(None, None, 0, None, None) == syn.ERR_INVALID
    assert c.syn_grad_clip(None, None, 0, 1.0, 1e-6, None, None) == syn.ERR_INVALID
    assert c.syn_grad_clip(None, None, 0, -1.0, 1e-6, None, None) == syn.ERR_INVALID


@pytest.mark.parametrize("kw, status", [
    (dict(d=0), syn.ERR_INVALID), (dict(d=-8), syn.ERR_INVALID), (dict(d=20), syn.ERR_UNSUPPORTED), (dict(d_ff=4), syn.ERR_UNSUPPORTED),
    (dict(d_ff=1 << 21), syn.ERR_UNSUPPORTED), (dict(dtype=2), syn.ERR_UNSUPPORTED), (dict(dtype=5), syn.ERR_INVALID),
    (dict(act=3), syn.ERR_INVALID), (dict(act=-1), syn.ERR_INVALID), (dict(backward=2), syn.ERR_INVALID),
    (dict(saved_f32=2), syn.ERR_INVALID)])
def test_refused_blocks(kw, status):
    c, h = ffn.FfnCfg(), ctypes.c_void_p()
    ffn.lib().syn_ffn_cfg_default(ctypes.byref(c))
    for k, v in kw.items():
        setattr(c, k, v)
    assert ffn.lib().syn_ffn_plan_create(ctypes.byref(h), ctypes.byref(c)) == status
    assert not h and syn.lib().syn_last_error()


@pytest.mark.parametrize("kw, status", [(dict(d=0), syn.ERR_INVALID), (dict(d=16385), syn.ERR_UNSUPPORTED), (dict(dtype=3), syn.ERR_INVALID)])
def test_refused_norms(kw, status):
    c, h = norm.NormCfg(), ctypes.c_void_p()
    norm.lib().syn_norm_cfg_default(ctypes.byref(c))
    for k, v in kw.items():
        setattr(c, k, v)
    assert norm.lib().syn_norm_plan_create(ctypes.byref(h), ctypes.byref(c)) == status
    assert not h and syn.lib().syn_last_error()


def test_headers_compile_as_plain_c(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "use_layer.c"
    src.write_text(
        '#include "syn_norm.h"\n#include "syn_ffn.h"\n#include "syn_clip.h"\n'
        "int use(void *x, float *f, void *stream) {\n"
        "    syn_norm_cfg_t nc;\n    syn_norm_plan_t np;\n    syn_ffn_cfg_t fc;\n    syn_ffn_plan_t fp;\n    syn_clip_plan_t cp;\n"
        "    if (syn_norm_cfg_default(&nc) || syn_ffn_cfg_default(&fc)) return -1;\n"
        "    fc.act = SYN_ACT_GELU_TANH;\n"
        "    if (syn_norm_plan_create(&np, &nc) || syn_ffn_plan_create(&fp, &fc) || syn_clip_plan_create(&cp)) return -1;\n"
        "    syn_norm_rows_t r = {x, 4096};\n    syn_ffn_mat_t m = {x, 14336};\n    syn_clip_tensor_t t = {x, x, 16, SYN_DTYPE_F32};\n"
        "    syn_layer_norm(np, &r, 0, 0, 1e-5f, &r, 4, stream);\n"
        "    syn_layer_norm_backward(np, &r, &r, 0, 1e-5f, &r, f, f, 4, stream);\n"
        "    syn_gated_ffn(fp, &m, &m, &m, &m, 0, 0, 4, stream);\n"
        "    syn_gated_ffn_backward(fp, &m, &m, &m, &m, &m, &m, &m, &m, 0, 0, 0, 4, stream);\n"
        "    syn_grad_norm(cp, &t, 1, f, stream);\n    syn_grad_clip(cp, &t, 1, 1.0f, 1e-6f, f, stream);\n"
        "    int st = syn_ffn_sync_status(fp, stream);\n"
        "    syn_norm_plan_destroy(np);\n    syn_ffn_plan_destroy(fp);\n    syn_clip_plan_destroy(cp);\n    return st;\n}\n")
    r = subprocess.run([gcc, "-std=c11", "-Wall", "-Werror", "-fsyntax-only", "-I", os.path.join(ROOT, "include"), str(src)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_parts_of_no_plan():
    n = ctypes.c_int(7)
    assert ffn.lib().syn_ffn_plan_parts(None, 1, 3, ctypes.byref(n), None) == syn.ERR_INVALID and n.value == 7
