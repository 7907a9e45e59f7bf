"""Host-only checks of the operators' C ABI (include/gemm_ops.h) and Python
binding: every declared function is exported, the ctypes mirrors list the
structs' fields in order, the header is valid C, and bad arguments are refused
before a GPU is touched."""
from __future__ import annotations

import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

import software_pipelined_tiled_gemm_gb300 as sg
from software_pipelined_tiled_gemm_gb300 import operators

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gemm_ops.h")
SOURCE = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


def test_library_exports_every_declared_symbol():
    names = sorted(set(re.findall(r"^[A-Za-z_][\w\s\*]*?\b(gemm_\w+)\s*\(", SOURCE, flags=re.M)))
    assert {"gemm_ops_create", "gemm_ffn_run", "gemm_ffn_backward", "gemm_orthogonalize",
            "gemm_token_logprobs", "gemm_token_logprobs_backward"} <= set(names)
    lib = sg.load_library()
    for n in names:
        assert ctypes.cast(getattr(lib, n), ctypes.c_void_p).value, n


@pytest.mark.parametrize("struct,mirror", [("gemm_ffn_args_t", sg.FfnArgs),
                                           ("gemm_orthogonalize_args_t", sg.OrthogonalizeArgs),
                                           ("gemm_logprobs_args_t", sg.LogprobsArgs)])
def test_struct_fields_match_the_header(struct, mirror):
    body = SOURCE[:SOURCE.index("} %s;" % struct)]
    body = body[body.rindex("typedef struct {") + len("typedef struct {"):]
    names = []
    for decl in body.split(";"):
        decl = decl.strip()
        if decl:
            names += [re.search(r"(\w+)\s*$", part).group(1) for part in decl.split(",")]
    assert names == [f[0] for f in mirror._fields_]


def test_max_top_k_matches_the_header():
    assert int(re.search(r"GEMM_LOGPROBS_MAX_TOP_K (\d+)", SOURCE).group(1)) == sg.MAX_TOP_K


def test_header_is_valid_c(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    (tmp_path / "h.c").write_text('#include "gemm_ops.h"\nint f(gemm_ops_t** o) { return (int)gemm_ops_create(o, 0); }\n')
    res = subprocess.run([cc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I",
                          os.path.join(ROOT, "include"), "-c", str(tmp_path / "h.c"), "-o",
                          str(tmp_path / "h.o")], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr


def test_null_and_negative_arguments_are_refused():
    lib = operators._lib()
    out = ctypes.c_void_p()
    assert lib.gemm_ops_create(None, 0) == sg.GEMM_ERR_INVALID_ARG
    assert lib.gemm_ops_create(ctypes.byref(out), -1) == sg.GEMM_ERR_INVALID_ARG and not out.value
    n = ctypes.c_size_t()
    a, g, p = sg.FfnArgs(), sg.OrthogonalizeArgs(), sg.LogprobsArgs()
    assert lib.gemm_ffn_workspace(None, ctypes.byref(a), 0, ctypes.byref(n)) == sg.GEMM_ERR_INVALID_ARG
    assert lib.gemm_ffn_run(None, ctypes.byref(a), None, 0, None) == sg.GEMM_ERR_INVALID_ARG
    assert lib.gemm_ffn_backward(None, ctypes.byref(a), None, 0, None) == sg.GEMM_ERR_INVALID_ARG
    assert lib.gemm_orthogonalize(None, ctypes.byref(g), None, 0, None) == sg.GEMM_ERR_INVALID_ARG
    assert lib.gemm_token_logprobs(None, ctypes.byref(p), None) == sg.GEMM_ERR_INVALID_ARG
    assert lib.gemm_token_logprobs_backward(None, ctypes.byref(p), None) == sg.GEMM_ERR_INVALID_ARG
    assert "NULL" in sg.gemm_last_error()
    d = ctypes.c_int32()
    assert lib.gemm_ops_check(None, ctypes.byref(d), None) == sg.GEMM_ERR_INVALID_ARG
    lib.gemm_ops_destroy(None)     # allowed, no-op


def test_kept_bytes():
    kept = operators._lib().gemm_ffn_kept_bytes
    assert kept(0, 64) == 0 and kept(64, 0) == 0
    # Two fp32 planes of whole 32-row blocks, then 16-bit rows of a multiple of 8.
    assert kept(1, 8) == 2 * 32 * 8 * 4 + 256
    assert kept(33, 5) == 2 * 64 * 5 * 4 + 33 * 8 * 2 + (-(33 * 8 * 2)) % 256


@pytest.mark.parametrize("call", [
    lambda t: sg.gated_ffn(t, t, t),
    lambda t: sg.orthogonalize(t),
    lambda t: sg.token_logprobs(t),
    lambda t: sg.token_logprobs_backward(t, None, None),
])
def test_cpu_tensors_and_other_objects_are_refused(call):
    with pytest.raises(ValueError, match="CUDA"):
        call(torch.zeros(4, 4))
    with pytest.raises(ValueError, match="CUDA"):
        call([[0.0]])


def test_unknown_activation_and_foreign_state_are_refused():
    t = torch.zeros(4, 4)
    with pytest.raises(ValueError, match="act"):
        sg.gated_ffn(t, t, t, act="tanh")
    with pytest.raises(TypeError, match="kept"):
        sg.gated_ffn_backward(t, t, t, t, kept=None)
