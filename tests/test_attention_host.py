"""The attention part of the C ABI without a GPU: struct layouts, constants,
refusals that need no device."""
import ctypes
import math
import os
import re
import subprocess

import pytest
import torch

from conftest import ROOT

HEADER = os.path.join(ROOT, "include", "mhc_attention.h")


@pytest.fixture(scope="module")
def capi():
    from mhc_residual_boundary_gb300 import build
    build.build()
    from mhc_residual_boundary_gb300 import capi as c
    c.lib()
    return c


def test_struct_layouts_match_the_header(capi, tmp_path):
    from mhc_residual_boundary_gb300 import attention
    structs = {"mhc_attention_config_t": capi.mhc_attention_config_t,
               "mhc_attention_append_args_t": capi.mhc_attention_append_args_t,
               "mhc_attention_attend_args_t": capi.mhc_attention_attend_args_t}
    packed = {"mhc_attention_append_args_t": attention.APPEND_ARGS, "mhc_attention_attend_args_t": attention.ATTEND_ARGS}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "mhc_attention.h"', "int main(void) {"]
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
    for name, st in packed.items():
        ct = structs[name]
        values = list(range(1, len(ct._fields_) + 1))
        raw = st.pack(*values)
        assert len(raw) <= ctypes.sizeof(ct)
        got = ct.from_buffer_copy(raw.ljust(ctypes.sizeof(ct), b"\0"))
        assert [getattr(got, f) for f, _ in ct._fields_] == values, name


def test_constants_match_the_header(capi):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    flags = {n: 1 << int(b) for n, b in re.findall(r"\b(MHC_ATTENTION_[A-Z0-9_]+)\s*=\s*1u\s*<<\s*(\d+)", text)}
    assert flags == {n: getattr(capi, n) for n in dir(capi) if n.startswith("MHC_ATTENTION_")}


def test_null_handles_fail_cleanly(capi):
    lib = capi.lib()
    for name, args in capi.ATTENTION_CALLS.items():
        assert getattr(lib, "mhc_attention_" + name)(None, ctypes.byref(args()), None) == 1
    assert lib.mhc_attention_check_errors(None) == 1
    assert lib.mhc_attention_destroy(None) == 0
    assert lib.mhc_attention_create(None, 0, None) == 1


@pytest.mark.parametrize("field,value,status", [
    ("heads", 0, "MHC_ERR_INVALID_ARG"), ("heads", 9, "MHC_ERR_INVALID_ARG"), ("heads", 4 * 129, "MHC_ERR_UNSUPPORTED"),
    ("kv_heads", 0, "MHC_ERR_INVALID_ARG"), ("kv_heads", -4, "MHC_ERR_INVALID_ARG"),
    ("head_dim", 96, "MHC_ERR_UNSUPPORTED"), ("page_size", 8, "MHC_ERR_UNSUPPORTED"),
    ("page_size", 48, "MHC_ERR_UNSUPPORTED"), ("rotary_dim", 8, "MHC_ERR_INVALID_ARG"),
    ("rotary_dim", -16, "MHC_ERR_INVALID_ARG"), ("rotary_dim", 144, "MHC_ERR_INVALID_ARG"),
    ("theta", 0.0, "MHC_ERR_INVALID_ARG"), ("theta", math.inf, "MHC_ERR_INVALID_ARG"),
    ("theta", math.nan, "MHC_ERR_INVALID_ARG"), ("flags", 1 << 2, "MHC_ERR_INVALID_ARG")])
def test_create_refuses_before_any_device_call(capi, field, value, status):
    c = capi.mhc_attention_config_t(16, 4, 128, 64, 128, 0, 10000.0, None)
    setattr(c, field, value)
    with pytest.raises(capi.MhcError, match=status):
        capi.mhc_attention_create(c, 0)


def test_frequencies_that_are_not_finite_are_refused(capi):
    f = (ctypes.c_double * 8)(*[1.0] * 7, math.nan)
    with pytest.raises(capi.MhcError, match="MHC_ERR_INVALID_ARG"):
        capi.mhc_attention_create(capi.mhc_attention_config_t(16, 4, 128, 64, 16, 0, 1.0, f), 0)


def test_the_wrapper_counts_frequencies(capi, monkeypatch):
    from mhc_residual_boundary_gb300 import attention
    made = []
    monkeypatch.setattr(attention.capi, "mhc_attention_create", lambda config, device: made.append((config, device)))
    with pytest.raises(ValueError, match="frequencies"):
        attention.Attention(heads=2, kv_heads=1, rotary_dim=32, frequencies=[1.0] * 15, device=0)
    a = attention.Attention(heads=2, kv_heads=1, rotary_dim=32, frequencies=torch.arange(16), device="cuda:1")
    (config, device), = made
    assert device == 1 and config.frequencies[15] == 15.0 and a.handle is None
    with pytest.raises(ValueError, match="CUDA device"):
        attention.Attention(heads=2, kv_heads=1, device="cpu")
