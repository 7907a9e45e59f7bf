"""Host-only checks of the grouped products, layer norm and AdamW: the ctypes
mirrors list the structs' fields in order, bad arguments are refused before a
GPU is touched, and what Python and C compute of sizes agrees."""
from __future__ import annotations

import ctypes
import os
import re
import struct

import pytest
import torch

import software_pipelined_tiled_gemm_gb300 as sg
from software_pipelined_tiled_gemm_gb300 import operators

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "gemm_ops.h")).read(), flags=re.S)


@pytest.mark.parametrize("name,mirror", [("gemm_grouped_args_t", sg.GroupedArgs),
                                         ("gemm_layer_norm_args_t", sg.LayerNormArgs),
                                         ("gemm_adamw_tensor_t", sg.AdamWTensor),
                                         ("gemm_adamw_args_t", sg.AdamWArgs)])
def test_struct_fields_match_the_header(name, mirror):
    body = SOURCE[:SOURCE.index("} %s;" % name)]
    body = body[body.rindex("typedef struct {") + len("typedef struct {"):]
    names = []
    for decl in body.split(";"):
        if decl.strip():
            names += [re.search(r"(\w+)\s*$", part.strip()).group(1) for part in decl.split(",")]
    assert names == [f[0] for f in mirror._fields_]


def test_constants_match_the_header():
    assert int(re.search(r"GEMM_GROUPED_MAX_GROUPS (\d+)", SOURCE).group(1)) == sg.MAX_GROUPS
    assert int(re.search(r"GEMM_ADAMW_BLOCK (\d+)", SOURCE).group(1)) == sg.ADAMW_BLOCK
    for name in ("GEMM_CHECK_OFFSETS", "GEMM_WAIT_NEXT_TILE", "GEMM_WAIT_NEXT_FREE"):
        role, n = re.search(r"%s \(\((\d) << 16\) \| (\d+)\)" % name, SOURCE).groups()
        text = sg.gemm_wait_detail_string(int(role) << 16 | int(n))
        assert text not in ("", "unknown wait"), name
        assert ("offsets" in text) == (name == "GEMM_CHECK_OFFSETS")


def test_table_of_tensors_has_the_struct_s_layout():
    assert operators._table(3).size == 3 * ctypes.sizeof(sg.AdamWTensor)
    packed = operators._table(1).pack(11, 12, 13, 14, 2, 1, 0, 0.5)
    t = sg.AdamWTensor.from_buffer_copy(packed)
    assert (t.param, t.grad, t.copy, t.numel, t.param_type, t.grad_type, t.copy_type, t.weight_decay) == (11, 12, 13, 14, 2, 1, 0, 0.5)
    assert struct.calcsize("P") == 8


def test_null_handles_are_refused():
    lib = operators._lib()
    n = ctypes.c_size_t()
    g, p, a = sg.GroupedArgs(), sg.LayerNormArgs(), sg.AdamWArgs()
    bad = sg.GEMM_ERR_INVALID_ARG
    assert lib.gemm_grouped_workspace(None, ctypes.byref(g), 0, ctypes.byref(n)) == bad
    assert lib.gemm_grouped_run(None, ctypes.byref(g), None, 0, None) == bad
    assert lib.gemm_grouped_backward(None, ctypes.byref(g), None, 0, None) == bad
    assert lib.gemm_layer_norm(None, ctypes.byref(p), None) == bad
    assert lib.gemm_layer_norm_backward_workspace(None, ctypes.byref(p), ctypes.byref(n)) == bad
    assert lib.gemm_layer_norm_backward(None, ctypes.byref(p), None, 0, None) == bad
    assert lib.gemm_adamw(None, ctypes.byref(a), None) == bad
    assert "NULL" in sg.gemm_last_error()


def test_state_elements():
    fn = operators._lib().gemm_adamw_state_elements
    fn.argtypes, fn.restype = [ctypes.c_void_p, ctypes.c_int64], ctypes.c_int64
    sizes = [1, 256, 257, 0, 1000]
    table = b"".join(operators._table(1).pack(0, 0, 0, s, 0, 0, 0, 0.0) for s in sizes)
    assert fn(ctypes.cast(table, ctypes.c_void_p), len(sizes)) == 256 + 256 + 512 + 0 + 1024
    assert fn(None, 0) == 0


@pytest.mark.parametrize("call", [
    lambda t: sg.grouped_matmul(t, t, t),
    lambda t: sg.grouped_matmul_backward(t, t, t, t),
    lambda t: sg.layer_norm(t),
    lambda t: sg.layer_norm_backward(t, t, None, sg.LayerNormKept(t, 4, 4, torch.float32)),
    lambda t: sg.adamw_state([t]),
    lambda t: sg.adamw([t], [t], sg.AdamWState(t, t, t, None), 1e-3),
])
def test_cpu_tensors_and_other_objects_are_refused(call):
    with pytest.raises(ValueError, match="CUDA"):
        call(torch.zeros(4, 4))
    with pytest.raises(ValueError, match="CUDA"):
        call([[0.0]])


def test_foreign_state_and_bad_choices_are_refused():
    t = torch.zeros(4, 4)
    with pytest.raises(TypeError, match="kept"):
        sg.layer_norm_backward(t, t, t, kept=None)
    with pytest.raises(ValueError, match="bits"):
        sg.adamw_state([t], bits=16)
    with pytest.raises(ValueError, match="at least one"):
        sg.adamw_state([])
