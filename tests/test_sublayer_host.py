"""The sublayer part of the C ABI without a GPU: struct layouts, constants,
refusals that need no device."""
import ctypes
import os
import re
import subprocess

import pytest

from conftest import ROOT

HEADER = os.path.join(ROOT, "include", "mhc_sublayer.h")


@pytest.fixture(scope="module")
def capi():
    from mhc_residual_boundary_gb300 import build
    build.build()
    from mhc_residual_boundary_gb300 import capi as c
    c.lib()
    return c


def test_struct_layouts_match_the_header(capi, tmp_path):
    from mhc_residual_boundary_gb300 import sublayer
    structs = {"mhc_sublayer_config_t": capi.mhc_sublayer_config_t,
               "mhc_sublayer_norm_args_t": capi.mhc_sublayer_norm_args_t,
               "mhc_sublayer_quantize_args_t": capi.mhc_sublayer_quantize_args_t,
               "mhc_sublayer_matmul_args_t": capi.mhc_sublayer_matmul_args_t,
               "mhc_sublayer_moe_args_t": capi.mhc_sublayer_moe_args_t}
    packed = {"mhc_sublayer_norm_args_t": sublayer.NORM_ARGS, "mhc_sublayer_quantize_args_t": sublayer.QUANTIZE_ARGS,
              "mhc_sublayer_matmul_args_t": sublayer.MATMUL_ARGS, "mhc_sublayer_moe_args_t": sublayer.MOE_ARGS}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "mhc_sublayer.h"', "int main(void) {"]
    for name, ct in structs.items():
        lines.append(f'printf("{name} size %zu\\n", sizeof({name}));')
        lines += [f'printf("{name} {f} %zu\\n", offsetof({name}, {f}));' for f, _ in ct._fields_]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["return 0; }"]))
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    for line in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines():
        name, field, value = line.split()
        ct = structs[name]
        assert int(value) == (ctypes.sizeof(ct) if field == "size" else getattr(ct, field).offset), line
    # the packed form: every field at its place, the last one included
    for name, st in packed.items():
        ct = structs[name]
        values = list(range(1, len(ct._fields_) + 1))
        raw = st.pack(*values)
        assert len(raw) <= ctypes.sizeof(ct)
        got = ct.from_buffer_copy(raw.ljust(ctypes.sizeof(ct), b"\0"))
        assert [getattr(got, f) for f, _ in ct._fields_] == values, name


def test_constants_match_the_header(capi):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    flags = {n: 1 << int(b) for n, b in re.findall(r"\b(MHC_SUBLAYER_[A-Z0-9_]+)\s*=\s*1u\s*<<\s*(\d+)", text)}
    assert flags == {n: getattr(capi, n) for n in dir(capi) if n.startswith("MHC_SUBLAYER_")}
    scores = {n: int(v) for n, v in re.findall(r"\b(MHC_SCORE_[A-Z]+)\s*=\s*(\d+)", text)}
    assert scores == {n: getattr(capi, n) for n in dir(capi) if n.startswith("MHC_SCORE_")}


def test_null_handles_fail_cleanly(capi):
    lib = capi.lib()
    for name, args in capi.SUBLAYER_CALLS.items():
        assert getattr(lib, "mhc_sublayer_" + name)(None, ctypes.byref(args()), None) == 1
    assert lib.mhc_sublayer_check_errors(None) == 1
    assert lib.mhc_sublayer_destroy(None) == 0
    assert lib.mhc_sublayer_create(None, 0, None) == 1


@pytest.mark.parametrize("field,value,status", [
    ("hidden", 250, "MHC_ERR_INVALID_ARG"), ("intermediate", 0, "MHC_ERR_INVALID_ARG"),
    ("hidden", 32768, "MHC_ERR_UNSUPPORTED"), ("num_experts", -1, "MHC_ERR_INVALID_ARG"),
    ("num_experts", 513, "MHC_ERR_UNSUPPORTED"), ("shared_experts", 9, "MHC_ERR_INVALID_ARG"),
    ("top_k", 0, "MHC_ERR_INVALID_ARG"), ("top_k", 17, "MHC_ERR_INVALID_ARG"),
    ("max_moe_tokens", 33, "MHC_ERR_INVALID_ARG"), ("score", 2, "MHC_ERR_INVALID_ARG"),
    ("flags", 1 << 3, "MHC_ERR_INVALID_ARG")])
def test_create_refuses_before_any_device_call(capi, field, value, status):
    c = capi.mhc_sublayer_config_t(256, 128, 32, 1, 4, 8, 0, 1.0, capi.MHC_SUBLAYER_FP8)
    setattr(c, field, value)
    with pytest.raises(capi.MhcError, match=status):
        capi.mhc_sublayer_create(c, 0)
