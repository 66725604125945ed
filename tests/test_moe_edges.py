"""CPU checks of the MoE operators' calls at the edges of their contracts: what they accept and refuse
before anything is launched."""
import ctypes
import os
import re
import subprocess

import pytest

import moe_grouped_gemm_02_gb300 as dg
from moe_grouped_gemm_02_gb300 import build as dg_build

GOOD = ctypes.c_void_p(0x10000)         # never dereferenced: every case returns before a launch
INVALID, OK = 1, 0


@pytest.fixture(scope="module")
def lib():
    dg_build.build()
    return dg.load_library()


def test_epilogue_calls_without_rows_take_null(lib):
    # tensors without elements have a null pointer; the weights, which have some, may not
    for b, sfb, want in ((GOOD, GOOD, OK), (None, GOOD, INVALID), (GOOD, None, INVALID)):
        assert lib.dg_fp8_gemm_nt_act(None, None, b, sfb, GOOD, None, None, None, 0, 512, 256, 4, 1, None) == want
        assert lib.dg_m_grouped_fp8_gemm_nt_contiguous_act(None, None, b, sfb, GOOD, None, None, None, None, 0, 512, 256, 4, 4, 1,
                                                           None) == want
        assert lib.dg_m_grouped_fp8_gemm_nt_masked_act(None, None, b, sfb, GOOD, None, None, None, GOOD, 4, 0, 512, 256, 4, 1,
                                                       None) == want
    assert lib.dg_m_grouped_fp8_gemm_nt_masked_act(None, None, GOOD, GOOD, None, None, None, None, None, 4, 0, 512, 256, 0, 0,
                                                   None) == INVALID      # masked_m has an entry per group
    # with rows every one of them is needed
    for hole in range(4):
        a, sfa, d, m = (None if i == hole else GOOD for i in range(4))
        assert lib.dg_m_grouped_fp8_gemm_nt_contiguous_act(a, sfa, GOOD, GOOD, None, None, None, d, m, 128, 512, 256, 4, 0, 0,
                                                           None) == INVALID


def test_activation_gradient_without_rows_takes_null(lib):
    for G in (1, 5):
        assert lib.dg_act_backward(None, None, None, None, None, None, 0, 256, G, 4, None) == OK
    assert lib.dg_act_backward(GOOD, GOOD, None, GOOD, None, None, 128, 256, 5, 4, None) == INVALID


def test_other_calls_of_the_layer_without_rows_take_null(lib):
    for b, want in ((GOOD, OK), (None, INVALID)):
        assert lib.dg_fp8_gemm_nt(None, None, b, GOOD, None, 0, 512, 256, None) == want
        assert lib.dg_m_grouped_fp8_gemm_nt_contiguous(None, None, b, GOOD, None, None, 0, 512, 256, 4, None) == want
        assert lib.dg_m_grouped_fp8_gemm_nt_masked(None, None, b, GOOD, None, GOOD, 4, 0, 512, 256, None) == want
        assert lib.dg_fp8_fp4_gemm_nt(None, None, b, GOOD, None, 0, 512, 256, None) == want
        assert lib.dg_m_grouped_fp8_fp4_gemm_nt_contiguous(None, None, b, GOOD, None, None, 0, 512, 256, 4, None) == want
        assert lib.dg_m_grouped_fp8_fp4_gemm_nt_masked(None, None, b, GOOD, None, GOOD, 4, 0, 512, 256, None) == want
        assert lib.dg_fp8_gemm(None, None, b, GOOD, None, None, 0, 512, 256, 0, 0, None) == want
    assert lib.dg_m_grouped_fp8_gemm_nt_contiguous(GOOD, GOOD, GOOD, GOOD, GOOD, None, 128, 512, 256, 4, None) == INVALID
    assert lib.dg_quantize_fp8_1x128(None, None, None, 4, 0, 256, None) == OK
    assert lib.dg_quantize_fp8_1x128(None, GOOD, GOOD, 1, 8, 256, None) == INVALID
    assert lib.dg_pack_sf_ue8m0(None, None, 1, 0, 256, 1, 128, None) == OK
    assert lib.dg_pack_sf_ue8m0_k_grouped(None, None, GOOD, 4, 64, 0, None) == OK
    assert lib.dg_pack_sf_ue8m0_k_grouped(None, GOOD, GOOD, 4, 64, 128, None) == INVALID
    k = lib.dg_k_grouped_fp8_gemm_tn_contiguous
    assert k(None, None, None, None, None, None, GOOD, 4, 0, 64, 0, None) == OK           # no columns of A either
    for hole in range(5):
        a, sfa, b, sfb, d = (None if i == hole else GOOD for i in range(5))
        assert k(a, sfa, b, sfb, None, d, GOOD, 4, 64, 64, 128, None) == INVALID


@pytest.mark.parametrize("source", ["dg_moe.cu", "dg_act.cu", "dg_quant.cu", "dg_pack.cu"])
def test_kernels_use_no_local_memory(source, tmp_path):
    # the compiler's report: no stack frame (an array indexed at run time) and no spilled registers
    cmd = [dg_build._nvcc(), *dg_build.GENCODE, *dg_build.FLAGS, "-Xptxas", "-v", "-c", os.path.join(dg_build.CSRC, source),
           "-o", str(tmp_path / "out.o")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    kernels = re.findall(r"Function properties for (\S+)\s+(\d+) bytes stack frame, (\d+) bytes spill stores, (\d+) bytes spill loads",
                         r.stdout + r.stderr)
    assert kernels
    assert [k for k in kernels if k[1:] != ("0", "0", "0")] == []


def test_host_tensors_are_refused():
    torch = pytest.importorskip("torch")
    dg_build.build()
    idx = torch.zeros((4, 2), dtype=torch.int32)
    with pytest.raises(TypeError, match="CUDA tensor"):
        dg.dg_moe_sort_masked(idx, idx, idx[:, 0].contiguous(), 8)
    with pytest.raises(TypeError, match="CUDA tensor"):
        dg.dg_act_backward(idx, idx, idx)


def test_launchers_keep_no_state_between_calls():
    # what belongs to a device is in the device's state (dg_api.cu), under its lock: the files with the kernels and their
    # launches have no variable of their own
    for name in sorted(os.listdir(dg_build.CSRC)):
        if name == "dg_api.cu" or not name.endswith((".cu", ".cuh")):
            continue
        text = open(os.path.join(dg_build.CSRC, name)).read()
        found = re.findall(r"^(?:static |inline |__device__ )*[\w:]+ \**g_\w+ *(?:=|;|\[).*$", text, re.M)
        assert found == [], name


def test_max_rows_of_sizes_past_an_int(lib):
    big = 1 << 32
    for T, k, G in ((big + 5, 1, 4), (5, big + 1, 4), (5, 1, big + 4), (1 << 31, 1, 4), (7 - big, 1, 4), (5, -1, 4)):
        assert dg.dg_moe_max_rows(T, k, G) == -1
    assert dg.dg_moe_max_rows(5, 2, 4) == 512
    assert dg.dg_moe_max_rows((1 << 31) - 1, 1, 1) == -1 and dg.dg_moe_max_rows((1 << 31) - 256, 1, 1) == (1 << 31) - 256


def test_a_build_that_failed_halfway_is_completed(tmp_path, monkeypatch):
    # the binding compiles, a kernel file does not: the next build links both anew.  (nvcc and g++ are stand-ins
    # that write their output files)
    src, out = tmp_path / "csrc", tmp_path / "out"
    src.mkdir(), out.mkdir()
    for name in ("one.cu", "two.cu", "dg_binding.cpp"):
        (src / name).write_text("first")
    nvcc = tmp_path / "nvcc"
    nvcc.write_text("""#!/bin/sh
log="$LOG"; prev=""; out=""
for a in "$@"; do
    [ "$prev" = "-o" ] && out="$a"
    case "$a" in *.cu) grep -q broken "$a" && exit 1;; esac
    prev="$a"
done
echo "$out" >> "$log"; touch "$out"
""")
    nvcc.chmod(0o755)
    log = tmp_path / "log"
    for k, v in {"CSRC": src, "INCLUDE": src, "BUILD_DIR": out, "LIB_PATH": out / "libdg.so", "BINDING_SRC": src / "dg_binding.cpp",
                 "BINDING_OBJ": out / "dg_binding.o", "BINDING_PATH": out / "dg_binding.so"}.items():
        monkeypatch.setattr(dg_build, k, str(v))
    monkeypatch.setenv("NVCC", str(nvcc))
    monkeypatch.setenv("LOG", str(log))

    def run(cmd, what):
        target = cmd[cmd.index("-o") + 1]
        with open(log, "a") as f:
            f.write(target + "\n")
        open(target, "w").close()
    monkeypatch.setattr(dg_build, "_run", run)

    def built():
        log.write_text("")
        dg_build.build()
        return {os.path.basename(x) for x in log.read_text().split()}

    assert built() == {"one.o", "two.o", "dg_binding.o", "libdg.so.tmp", "dg_binding.so.tmp"}
    assert built() == set()
    past = os.stat(out / "dg_binding.so").st_mtime - 100         # everything so far is old; then two files change
    for p in list(src.iterdir()) + list(out.iterdir()):
        os.utime(p, (past, past))
    (src / "dg_binding.cpp").write_text("second")
    (src / "two.cu").write_text("broken")
    with pytest.raises(RuntimeError):
        built()
    (src / "two.cu").write_text("second")
    assert built() == {"two.o", "libdg.so.tmp", "dg_binding.so.tmp"}
    assert built() == set()


def test_words_across_a_word_boundary_are_refused(lib):
    # int32 and float32 tensors at an address that is no multiple of 4: a read of one would fault
    half, align = ctypes.c_void_p(0x10002), 3
    bad = [lib.dg_moe_sort(half, GOOD, GOOD, GOOD, None, 8, 2, 4, 512, None), lib.dg_moe_sort(GOOD, half, GOOD, GOOD, None, 8, 2, 4, 512, None),
           lib.dg_moe_sort(GOOD, GOOD, GOOD, half, None, 8, 2, 4, 512, None), lib.dg_moe_sort(GOOD, GOOD, GOOD, GOOD, half, 8, 2, 4, 512, None),
           lib.dg_moe_sort_masked(half, GOOD, GOOD, 8, 2, 4, 16, None), lib.dg_moe_sort_masked(GOOD, GOOD, half, 8, 2, 4, 16, None),
           lib.dg_moe_dispatch(GOOD, half, None, GOOD, 8, 2, 256, 128, 0, None),
           lib.dg_moe_dispatch_fp8(GOOD, half, None, GOOD, GOOD, 8, 2, 256, 1, 128, None),
           lib.dg_moe_combine(GOOD, half, None, None, GOOD, 8, 2, 256, 128, 0, None),
           lib.dg_moe_combine(GOOD, GOOD, half, None, GOOD, 8, 2, 256, 128, 0, None),
           lib.dg_moe_combine_backward(GOOD, GOOD, GOOD, None, half, GOOD, GOOD, 8, 2, 256, 128, 0, None),
           lib.dg_moe_combine_backward(GOOD, GOOD, GOOD, None, GOOD, GOOD, half, 8, 2, 256, 128, 0, None),
           lib.dg_m_grouped_fp8_gemm_nt_contiguous_act(GOOD, GOOD, GOOD, GOOD, None, None, None, GOOD, half, 128, 512, 256, 4, 0, 0, None),
           lib.dg_m_grouped_fp8_gemm_nt_masked_act(GOOD, GOOD, GOOD, GOOD, None, None, None, GOOD, half, 4, 64, 512, 256, 0, 0, None),
           lib.dg_m_grouped_fp8_gemm_nt_contiguous(GOOD, GOOD, GOOD, GOOD, GOOD, half, 128, 512, 256, 4, None),
           lib.dg_k_grouped_fp8_gemm_tn_contiguous(GOOD, GOOD, GOOD, GOOD, None, GOOD, half, 4, 64, 64, 128, None),
           lib.dg_pack_sf_ue8m0_k_grouped(GOOD, GOOD, half, 4, 64, 128, None)]
    assert bad == [align] * len(bad)
