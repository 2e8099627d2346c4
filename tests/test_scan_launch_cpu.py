"""CPU checks of the selective scan's host side: which form a batch takes for what the runtime
reports of its kernels (a fake runtime, nothing is launched), how much memory a call asks for, which
sizes the binding refuses, and the softplus series' error."""
import ctypes
import os
import re
import shutil
import subprocess

import numpy as np
import pytest

import invariant_linear_attention_gb300 as gdn
from invariant_linear_attention_gb300 import binding, build_lib

FAKE = 0x10000  # never dereferenced: the fake runtime launches nothing
OK, CUDA_ERROR = 0, -4

RUNTIME = r"""
#include <cuda_runtime_api.h>
#include <string.h>
#include <map>
#include <string>
static std::map<const void*, std::string>& names() { static std::map<const void*, std::string> m; return m; }
static std::string last;
extern "C" {
int fake_regs = 0, fake_error = 0, fake_asked = 0;
const char* fake_last() { return last.c_str(); }
void** __cudaRegisterFatBinary(void*) { static void* h; return &h; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char* host, char*, const char* name, int, void*, void*, void*, void*, int*) { names()[host] = name; }
unsigned __cudaPushCallConfiguration(dim3, dim3, size_t, void*) { return 0; }
cudaError_t __cudaPopCallConfiguration(dim3* g, dim3* b, size_t* s, void* st) { return *g = *b = dim3{1, 1, 1}, *s = 0, *static_cast<void**>(st) = 0, cudaSuccess; }
cudaError_t __cudaGetKernel(void** k, const void* host) { return *k = const_cast<void*>(host), cudaSuccess; }
cudaError_t __cudaLaunchKernel(void* k, dim3, dim3, void**, size_t, void*) { return last = names()[k], cudaSuccess; }
cudaError_t CUDARTAPI cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t CUDARTAPI cudaGetLastError() { return cudaSuccess; }
cudaError_t CUDARTAPI cudaFuncGetAttributes(cudaFuncAttributes* a, const void*) {
    memset(a, 0, sizeof *a);
    ++fake_asked;
    return a->numRegs = fake_regs, static_cast<cudaError_t>(fake_error);
}
}
"""


@pytest.fixture(scope="module")
def faked(tmp_path_factory):
    """A function that loads the scan's forward on a fresh copy of the fake runtime."""
    build_lib.build()
    obj = os.path.join(build_lib.BUILD, "gdn_scan.o")
    nvcc = build_lib._nvcc()
    if not os.path.exists(obj):
        os.makedirs(build_lib.BUILD, exist_ok=True)
        build_lib._compile(nvcc, os.path.join(build_lib.CSRC, "gdn_scan.cu"))
    at = tmp_path_factory.mktemp("fake")
    (at / "runtime.cpp").write_text(RUNTIME)
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-Wl,-Bsymbolic", "-I" + include, str(at / "runtime.cpp"), obj, "-o", str(at / "scan.so")], check=True)
    count = [0]

    def load():
        count[0] += 1
        shutil.copy(at / "scan.so", at / f"scan{count[0]}.so")
        L = ctypes.CDLL(str(at / f"scan{count[0]}.so"))
        L.gdn_selective_scan_fwd.argtypes = [ctypes.POINTER(gdn.ScanShape)] + [ctypes.c_void_p] * 11 + [ctypes.c_int] + [ctypes.c_void_p] * 3
        L.fake_last.restype = ctypes.c_char_p
        return L

    return load


def forward(L, S, blocks):
    """Status of a prompt of `blocks` CTAs of one channel a lane, and the channels a lane of the form it took."""
    C = blocks * (64 if S <= 16 else 1024 // S)
    s = gdn.ScanShape(N=1, T_total=100, C=C, G=1, S=S, dtype=binding.GDN_BF16, dt_softplus=1, ldx=C, lddt=C, ldz=C, ldB=S, ldC=S)
    p = [FAKE + 0x1000 * i for i in range(12)]
    st = L.gdn_selective_scan_fwd(ctypes.byref(s), *p[:9], None, None, 0, None, p[10], None)
    name = L.fake_last().decode()
    assert st != OK or f"scan_fwd_kernelI13__nv_bfloat16Li{S}ELi" in name
    return st, name.split(f"Li{S}ELi")[1][0] if st == OK else None


def regs(L, n, error=0):
    ctypes.c_int.in_dll(L, "fake_regs").value = n
    ctypes.c_int.in_dll(L, "fake_error").value = error


@pytest.mark.parametrize("S", [16, 32, 64])
def test_full_batches_do_without_registers_to_move(faked, S):
    L = faked()
    regs(L, 80)
    assert forward(L, S, 100) == (OK, "1") and forward(L, S, 1000) == (OK, "2")
    # a kernel compiled to fewer registers than its warpgroups would own: the other form, which has the same bits
    L = faked()
    regs(L, 79)
    for _ in range(3):
        assert forward(L, S, 1000) == (OK, "1")
    assert ctypes.c_int.in_dll(L, "fake_asked").value == 1
    # an error of the runtime is an error, and is not remembered
    L = faked()
    regs(L, 80, error=2)
    assert forward(L, S, 1000)[0] == CUDA_ERROR
    regs(L, 80)
    assert forward(L, S, 1000) == (OK, "2")


def workspace(N, T, C, S, G=1, dtype=binding.GDN_BF16):
    build_lib.build()
    s = gdn.ScanShape(N=N, T_total=T, C=C, G=G, S=S, dtype=dtype, dt_softplus=1, ldx=C, lddt=C, ldz=C, ldB=G * S, ldC=G * S)
    return gdn.lib().gdn_selective_scan_bwd_workspace_size(ctypes.byref(s))


@pytest.mark.parametrize("T,C,S,G", [(8192, 4096, 16, 1), (32768, 8192, 16, 1), (8192, 1024, 64, 2), (300, 64, 8, 1), (5, 64, 8, 1)])
@pytest.mark.parametrize("N", [1, 8, 256, 1024, 4096])
def test_scan_backward_workspace_follows_the_tokens_and_the_sequences(T, C, S, G, N):
    """A state every 8 tokens, two per segment (never more than T / 16 + N), dB and dC per block of channels."""
    segs, blocks = T // 16 + N, G * -(-(C // G) // (64 if S <= 16 else 32))
    bound = 4 * (C * S + C) * (T // 8) + 4 * (2 * C * S + 3 * C) * segs + 8 * S * T * blocks
    assert 0 < workspace(N, T, C, S, G) <= bound
    assert workspace(N + 1000, T, C, S, G) - workspace(N, T, C, S, G) <= 1000 * 4 * (2 * C * S + 3 * C) + 4 * (2 * C * S + 3 * C) * (T // 16)


def test_scan_backward_workspace_of_many_short_documents():
    # 64 MB of bf16 x: states of 4096 sequences are 1 GB, twice in the workspace
    assert workspace(4096, 8192, 4096, 16) < 2.8e9
    assert workspace(8, 8192, 4096, 16) < 0.45e9


@pytest.mark.parametrize("kind,values", [
    (gdn.ConvShape, (1, 2 ** 32 + 5, 8, 4, binding.GDN_BF16, 1)), (gdn.ConvShape, (1, 2 ** 31, 8, 4, binding.GDN_BF16, 1)),
    (gdn.ScanShape, (1, 2 ** 32 + 5, 8, 1, 8, binding.GDN_BF16, 1, 8, 8, 8, 8, 8)), (gdn.ScanShape, (2 ** 32, 0, 8, 1, 8, binding.GDN_BF16, 1, 8, 8, 8, 8, 8)),
    (gdn.QkShape, (5, 2 ** 32 + 2, 2, 64, 32, 0, 0, 100, 1e-6, binding.GDN_BF16, 2 ** 40, 128)),
    (gdn.QkShape, (5, 2, 2, 64, 32, 0, 0, 2 ** 32 + 100, 1e-6, binding.GDN_BF16, 128, 128))])
def test_sizes_past_the_structs_integers_are_refused(kind, values):
    """A tensor of 2^32 + 5 rows is not one of 5."""
    with pytest.raises(ValueError):
        binding._struct(kind, *values)


def test_large_sizes_within_the_structs_integers_are_not():
    binding._struct(gdn.QkShape, 2 ** 40, 2, 2, 64, 32, 0, 0, 2 ** 31 - 1, 1e-6, binding.GDN_BF16, 2 ** 40, 128)
    binding._struct(gdn.ScanShape, 1, 2 ** 31 - 1, 8, 1, 8, binding.GDN_BF16, 1, 2 ** 33, 8, 8, 8, 8)


def test_softplus_series_error():
    """The kernels' polynomial for 2 artanh(w) / w in w^2 on [0, 1/9], as committed, in 64 bits: within 8e-9."""
    with open(os.path.join(build_lib.CSRC, "gdn_scan.cuh")) as f:
        body = f.read().split("float2 softplus2")[1].split("return")[0]
    c = [float(v) for v in re.findall(r"both\((\d\.\d+)f\)", body)] + [2.0]
    assert len(c) == 5 and "__ffma2_rn(p, q, both(2.f))" in body
    w = np.linspace(1e-4, 1 / 3, 100001)
    series = 2 * np.arctanh(w) / w
    assert np.abs(np.polyval(c, w * w) / series - 1).max() < 8e-9
