"""libgemm_layers.h on the CPU: exports, sizes, every refusal (no call here
reaches a kernel launch), the choice of kernels, and the reference's own
definitions."""
import os
import re
import subprocess
import sys

import pytest
import torch

import layers_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "libgemm_layers.h")


@pytest.fixture(scope="module")
def lib():
    from dense_gemm_optimisation_amd import binding
    if not os.path.exists(binding.LIB_PATH):
        from dense_gemm_optimisation_amd import build
        build.build()
    return binding


def test_every_declared_symbol_is_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(gemm_\w+)\s*\(", text)))
    out = subprocess.run(["nm", "-D", "--defined-only", lib.LIB_PATH], capture_output=True, text=True, check=True).stdout
    exported = set(re.findall(r"\bT (\w+)$", out, flags=re.M))
    assert len(names) == 12
    for name in names:
        assert name in exported, name
        assert getattr(lib.library(), name).argtypes is not None


def test_header_compiles_as_c(tmp_path):
    src = tmp_path / "use.c"
    src.write_text('#include "libgemm_layers.h"\nint f(void){return GEMM_WEIGHTS_E5M2 + GEMM_ACT_SILU;}\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    "-I" + os.path.dirname(HEADER), "-c", str(src), "-o", str(tmp_path / "use.o")], check=True)


# ---- the reference's definitions
@pytest.mark.parametrize("a", ["none", "relu", "gelu", "silu"])
def test_reference_slopes_against_differences(a):
    z = torch.linspace(-6, 6, 241, dtype=torch.float64) + 0.0123  # off ReLU's corner
    h = 1e-5
    d = (ref.act(z + h, a) - ref.act(z - h, a)) / (2 * h)
    # h^2 times a third derivative of at most 2, and 64-bit rounding over h
    assert ((d - ref.slope(z, a)).abs() < 1e-9).all()


def test_reference_steps_on_a_diagonal():
    s = torch.tensor([1.0, 0.5, 0.25, 0.01], dtype=torch.float64)
    x = ref.newton_schulz(torch.diag(s), 2)
    s = s / s.norm()
    for _ in range(2):
        s = 3.4445 * s - 4.7750 * s ** 3 + 2.0315 * s ** 5
    assert (x - torch.diag(s)).abs().max() < 1e-14


# ---- refusals: addresses that are never followed
A, B, BIAS, R, C, Z, W, DB = (i << 36 for i in range(1, 9))


def linear_call(lib, names=False, **k):
    d = dict(M=64, N=96, K=200, alpha=1.0, A=A, lda=200, B=B, ldb=200, order_b=1, in_type=1, bias=BIAS, act=2, beta=1.0, R=R,
             ldr=96, C=C, ldc=96, type_c=1, Z=Z, ldz=96, workspace=W, workspace_bytes=1 << 30)
    d.update(k)
    return lib.linear_kernel_name(**d) if names else lib.gemm_linear(**d, raise_on_error=False)


@pytest.mark.parametrize("bad", [
    dict(M=-1), dict(N=-1), dict(K=-1), dict(A=0), dict(B=0), dict(C=0), dict(R=0), dict(A=A + 1), dict(B=B + 1), dict(C=C + 1),
    dict(R=R + 1), dict(Z=Z + 1), dict(bias=BIAS + 1), dict(lda=199), dict(ldb=199), dict(order_b=0, ldb=95), dict(order_b=2),
    dict(ldc=95), dict(ldr=95), dict(ldz=95), dict(ldc=-1), dict(in_type=0), dict(in_type=3), dict(type_c=2), dict(type_c=3),
    dict(act=4), dict(act=-1), dict(C=A), dict(C=B + 64), dict(C=R + 2), dict(C=R, ldc=97), dict(C=BIAS), dict(C=Z), dict(Z=R),
    dict(Z=A + 2), dict(workspace=W + 8), dict(workspace=0), dict(workspace=C), dict(workspace=A), dict(type_c=0, C=R, Z=R + 8),
    dict(M=1 << 41), dict(M=1 << 39, N=1 << 39), dict(lda=1 << 41), dict(workspace=BIAS),
])
def test_linear_refuses(lib, bad):
    assert linear_call(lib, **bad) == lib.ERR_INVALID_ARG
    assert linear_call(lib, names=True, **bad) is None


def test_linear_empty(lib):
    for empty in (dict(M=0), dict(N=0)):
        assert linear_call(lib, **empty, A=0, C=0, B=0) == lib.OK
        assert linear_call(lib, names=True, **empty, A=0, C=0) == ""
    with pytest.raises(lib.GemmError):
        lib.gemm_linear(-1, 1, 1, 1.0, A, 1, B, 1, 1, 1, 0, 0, 0.0, 0, 0, C, 1, 1)


def backward_call(lib, names=False, **k):
    d = dict(M=64, N=96, K=200, alpha=1.0, A=A, lda=200, B=B, ldb=200, order_b=1, in_type=2, Z=Z, ldz=96, act=3, D=C, ldd=96,
             type_d=2, beta=0.0, d_bias=DB, workspace=W, workspace_bytes=1 << 30)
    d.update(k)
    return lib.linear_backward_kernel_name(**d) if names else lib.gemm_linear_backward(**d, raise_on_error=False)


@pytest.mark.parametrize("bad", [
    dict(M=-1), dict(N=-1), dict(K=-1), dict(A=0), dict(B=0), dict(D=0), dict(Z=0), dict(Z=Z + 1), dict(D=C + 1), dict(ldz=95),
    dict(ldd=95), dict(lda=199), dict(ldb=199), dict(in_type=0), dict(type_d=1), dict(act=4), dict(D=A), dict(D=B), dict(D=Z + 2),
    dict(D=Z, ldd=97), dict(D=Z, type_d=0), dict(d_bias=DB + 2), dict(d_bias=C + 4), dict(d_bias=Z + 4), dict(d_bias=A),
    dict(workspace=0, workspace_bytes=0), dict(workspace_bytes=700), dict(workspace=W + 4), dict(workspace=DB), dict(workspace=Z),
])
def test_linear_backward_refuses(lib, bad):
    assert backward_call(lib, **bad) == lib.ERR_INVALID_ARG
    assert backward_call(lib, names=True, **bad) is None


def test_linear_backward_empty(lib):
    assert backward_call(lib, M=0, d_bias=0, A=0, D=0) == lib.OK
    assert backward_call(lib, N=0, A=0, D=0) == lib.OK
    assert backward_call(lib, M=0, d_bias=DB + 1) == lib.ERR_INVALID_ARG


def activation_call(lib, **k):
    d = dict(M=64, N=96, A=A, lda=96, type_a=1, Z=Z, ldz=96, type_z=1, act=2, D=C, ldd=96, type_d=1, beta=0.0, d_bias=DB,
             workspace=W, workspace_bytes=1 << 20)
    d.update(k)
    return lib.gemm_activation_backward(**d, raise_on_error=False)


@pytest.mark.parametrize("bad", [
    dict(M=-1), dict(N=-1), dict(A=0), dict(A=A + 1), dict(type_a=0, A=A + 2), dict(lda=95), dict(type_a=3), dict(type_z=-1),
    dict(Z=0), dict(Z=Z + 1), dict(ldz=95), dict(act=4), dict(D=0, d_bias=0), dict(D=C + 1), dict(ldd=95), dict(type_d=3),
    dict(D=A + 2), dict(D=A, type_d=2), dict(D=A, ldd=97), dict(D=Z + 2), dict(D=Z, type_d=0), dict(d_bias=DB + 1), dict(d_bias=A),
    dict(d_bias=C), dict(workspace=0), dict(workspace=W + 8), dict(workspace_bytes=10), dict(workspace=A), dict(workspace=C),
    dict(M=1 << 39, N=1 << 39),
])
def test_activation_backward_refuses(lib, bad):
    assert activation_call(lib, **bad) == lib.ERR_INVALID_ARG


def test_activation_backward_empty(lib):
    assert activation_call(lib, N=0, A=0) == lib.OK
    assert activation_call(lib, M=0, A=0, d_bias=0) == lib.OK
    assert activation_call(lib, M=0, d_bias=DB + 2) == lib.ERR_INVALID_ARG
    n = (1 << 28) + 1
    assert activation_call(lib, M=1, N=n, lda=n, ldz=n, ldd=n, D=0, Z=Z, workspace_bytes=1 << 31) == lib.ERR_UNSUPPORTED


def layer_call(lib, **k):
    d = dict(tokens=8, experts=16, top_k=2, D=200, H=72, X=A, ldx=200, in_type=1, ids=R, weights=R + 4096, type_w=0, up=B,
             ld_up=200, stride_up=144 * 200, scale_up=0, lds_up=0, stride_scale_up=0, down=BIAS, ld_down=72, stride_down=200 * 72,
             scale_down=0, lds_down=0, stride_scale_down=0, act=3, beta=0.0, Y=C, ldy=200, type_y=1, workspace=W,
             workspace_bytes=1 << 20)
    d.update(k)
    return lib.gemm_experts_layer(**d, raise_on_error=False)


CODES = dict(type_w=1, ld_up=208, stride_up=144 * 208, scale_up=Z, lds_up=2, stride_scale_up=4, ld_down=80, stride_down=200 * 80,
             scale_down=Z + 4096, lds_down=2, stride_scale_down=2)


@pytest.mark.parametrize("bad", [
    dict(tokens=-1), dict(experts=0), dict(top_k=0), dict(top_k=17), dict(D=-1), dict(H=-1), dict(H=0), dict(X=0), dict(X=A + 8),
    dict(ldx=199), dict(ldx=204), dict(ldx=192), dict(in_type=0), dict(ids=0), dict(ids=R + 2), dict(weights=0),
    dict(weights=R + 4097), dict(type_w=3), dict(type_w=-1), dict(type_w=1), dict(up=0), dict(up=B + 8), dict(ld_up=192),
    dict(ld_up=201), dict(stride_up=4), dict(stride_up=-8), dict(down=0), dict(down=BIAS + 2), dict(ld_down=64), dict(ld_down=73),
    dict(stride_down=3), dict(act=0), dict(act=4), dict(Y=0), dict(Y=C + 1), dict(ldy=199), dict(type_y=2), dict(workspace=0),
    dict(workspace=W + 8), dict(workspace_bytes=8 * 2 * 72 * 4), dict(Y=A), dict(Y=B + 16), dict(Y=BIAS), dict(Y=W), dict(Y=R),
    dict(workspace=A), dict(workspace=B), dict(workspace=R), dict(D=1 << 41),
    dict(CODES, scale_up=0), dict(CODES, scale_down=Z + 2), dict(CODES, lds_up=1), dict(CODES, lds_down=1, H=200, ld_down=208),
    dict(CODES, ld_up=200), dict(CODES, stride_up=8), dict(CODES, stride_scale_up=-1), dict(CODES, Y=Z), dict(CODES, workspace=Z),
])
def test_experts_layer_refuses(lib, bad):
    assert layer_call(lib, **bad) == lib.ERR_INVALID_ARG


def test_experts_layer_empty_and_unsupported(lib):
    assert layer_call(lib, tokens=0, X=0) == lib.OK
    assert layer_call(lib, D=0, X=0) == lib.OK
    assert layer_call(lib, tokens=65) == lib.ERR_UNSUPPORTED
    assert layer_call(lib, experts=1025) == lib.ERR_UNSUPPORTED
    assert layer_call(lib, experts=64, top_k=33) == lib.ERR_UNSUPPORTED


def ortho_call(lib, **k):
    d = dict(M=40, N=30, G=A, ldg=30, in_type=1, steps=5, coefficients=None, eps=1e-7, alpha=1.0, beta=0.0, O=C, ldo=30, type_o=0,
             workspace=W, workspace_bytes=1 << 24)
    d.update(k)
    return lib.gemm_orthogonalize(**d, raise_on_error=False)


@pytest.mark.parametrize("bad", [
    dict(M=-1), dict(N=-1), dict(batch=-1), dict(G=0), dict(G=A + 1), dict(ldg=29), dict(in_type=3), dict(type_o=-1), dict(steps=0),
    dict(steps=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(O=0), dict(O=C + 2), dict(ldo=29),
    dict(O=A), dict(workspace=0), dict(workspace=W + 8), dict(workspace_bytes=1000), dict(workspace=A), dict(workspace=C),
    dict(batch=2, stride_g=1200, stride_o=1199), dict(batch=2, stride_g=-1, stride_o=1200), dict(M=1 << 41),
    dict(M=1 << 39, N=1 << 39), dict(batch=1 << 39, stride_o=1200),
])
def test_orthogonalize_refuses(lib, bad):
    assert ortho_call(lib, **bad) == lib.ERR_INVALID_ARG


def test_orthogonalize_empty_and_unsupported(lib):
    for empty in (dict(M=0), dict(N=0), dict(batch=0)):
        assert ortho_call(lib, **empty, G=0, O=0) == lib.OK
    assert ortho_call(lib, steps=33) == lib.ERR_UNSUPPORTED
    assert ortho_call(lib, M=1, N=1 << 21, ldg=1 << 21, ldo=1 << 21, workspace_bytes=1 << 34) == lib.ERR_UNSUPPORTED
    with pytest.raises(ValueError):
        lib.gemm_orthogonalize(4, 4, A, 4, 0, 2, [(1.0, 2.0, 3.0)], 0.0, 1.0, 0.0, C, 4, 0, W, 1 << 20)


# ---- sizes and names
def test_sizes(lib):
    assert lib.linear_workspace_size(-1, 4, 4) == 0 and lib.linear_workspace_size(0, 4, 4) == 0
    assert lib.linear_workspace_size(16, 4096, 4096) >= 16 * 4096 * 4
    assert lib.activation_backward_workspace_size(-1, 4) == 0
    assert lib.activation_backward_workspace_size(1, 4) >= 16
    assert lib.experts_layer_workspace_size(65, 8, 2, 64, 64) == 0
    assert lib.experts_layer_workspace_size(64, 8, 2, 64, 64) >= 64 * 2 * 64 * 4
    assert lib.orthogonalize_workspace_size(0, 4, 1) == 0
    assert lib.orthogonalize_workspace_size(100, 50, 2) >= 2 * (3 * 50 * 104 + 2 * 50 * 56) * 2


def test_orthogonalize_too_large_to_launch(lib):
    """2^24 blocks of 64 x 64 of a matrix are refused before anything is launched (a call that got past the checks would end in
    ERR_HIP here, without a GPU)."""
    most = lib.orthogonalize_workspace_size(1 << 20, 1 << 16, 1)
    for M, N in ((1 << 20, 1 << 16), (1 << 16, 1 << 20), ((1 << 20) - 63, (1 << 16) - 63)):
        assert ortho_call(lib, M=M, N=N, ldg=N, ldo=N, G=1 << 50, O=1 << 52, workspace=1 << 54,
                          workspace_bytes=most) == lib.ERR_UNSUPPORTED


# ---- the device that a call configures its kernels on
RECORDER = r"""
#include <stdio.h>
#include <stddef.h>
typedef struct { unsigned x, y, z; } dim3_t;
static int current = 0;
int hipGetDevice(int *d) { *d = current; return 0; }
int hipSetDevice(int d) { current = d; return 0; }
int hipStreamGetDevice(void *stream, int *d) { *d = stream ? 1 : current; return 0; }
int hipFuncSetAttribute(const void *f, int a, int v) { printf("attribute %d\n", current); fflush(stdout); return 0; }
int hipLaunchKernel(const void *f, dim3_t g, dim3_t b, void **p, size_t lds, void *stream) {
    printf("launch %d\n", lds > 65536); fflush(stdout); return 0;
}
static dim3_t grid, block;
static size_t dynamic;
static void *on;
int __hipPushCallConfiguration(dim3_t g, dim3_t b, size_t lds, void *stream) {
    grid = g; block = b; dynamic = lds; on = stream; return 0;
}
int __hipPopCallConfiguration(dim3_t *g, dim3_t *b, size_t *lds, void **stream) {
    *g = grid; *b = block; *lds = dynamic; *stream = on; return 0;
}
int hipGetLastError(void) { return 0; }
"""


@pytest.mark.parametrize("stream,device", [(0, 0), (0x1000, 1)])
def test_large_lds_is_allowed_on_the_streams_device(lib, tmp_path, stream, device):
    """A kernel of more than 64 KiB of dynamic LDS is allowed them where it runs: on the device of `stream`, which need not be
    the current one (and that stays current).  HIP's calls are recorded, nothing runs."""
    src, so = tmp_path / "recorder.c", tmp_path / "recorder.so"
    src.write_text(RECORDER)
    subprocess.run(["gcc", "-shared", "-fPIC", str(src), "-o", str(so)], check=True)
    call = f"""
import ctypes, sys
recorder = ctypes.CDLL({str(so)!r}, mode=ctypes.RTLD_GLOBAL)  # before HIP's own library: its names are found first
sys.path.insert(0, {ROOT!r})
from dense_gemm_optimisation_amd import binding as lib
p = [i << 36 for i in range(1, 9)]
print("begin", flush=True)
lib.gemm_orthogonalize(128, 128, p[0], 128, 0, 5, None, 0.0, 1.0, 0.0, p[1], 128, 0, p[2], 1 << 30, stream={stream})
lib.gemm_experts_layer(1, 64, 8, 4096, 1024, p[0], 4096, 1, p[1], p[2], 0, p[3], 4096, 2048 * 4096, 0, 0, 0, p[4], 1024, 4096 * 1024,
                       0, 0, 0, 3, 0.0, p[5], 4096, 1, p[6], 1 << 30, stream={stream})
d = ctypes.c_int(-1)
recorder.hipGetDevice(ctypes.byref(d))
print("current", d.value, flush=True)
"""
    out = subprocess.run([sys.executable, "-c", call], capture_output=True, text=True, check=True).stdout
    said = out.split("begin\n")[1].splitlines()
    assert said == [f"attribute {device}", "launch 1"] * 3 + ["current 0"]


@pytest.mark.parametrize("M,N,K,odd,split", [
    (64, 512, 512, 0, True), (64, 512, 256, 0, False), (64, 4096, 1024, 0, True), (768, 1024, 1024, 0, False),
    (1024, 1024, 1024, 0, False), (1024, 1024, 4096, 0, True), (1024, 2048, 1024, 0, False), (2048, 2048, 512, 0, False),
    (2048, 2048, 2048, 0, False), (2048, 2048, 16384, 0, True), (64, 512, 256, 1, True), (1000, 1024, 512, 1, False),
    (1000, 1024, 1024, 1, True), (900, 2048, 1024, 1, False), (900, 2048, 4096, 1, True),
])
def test_linear_cuts_k_where_that_pays(lib, M, N, K, odd, split):
    """K in slices costs a second launch and the sums' way through memory: not for few steps of K, and the fewer the more tiles
    there are."""
    name = linear_call(lib, names=True, M=M, N=N, K=K, lda=K + odd, ldb=K + odd, ldc=N, ldr=N, ldz=N)
    kernel = "linear_mfma_any" if odd else "linear_mfma_128"
    assert name == kernel + ("_split" if split else "")
