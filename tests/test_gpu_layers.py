"""libgemm_layers.h on the GPU against its definitions in 64 bits.

The bounds are layers_reference.py's: fp32 sums in any order, the activations'
relative errors, one rounding of each output.  Newton-Schulz steps amplify
their roundings in ways that no short bound follows, so their tolerance is
twice what the same roundings do to the same matrix in 64 bits (see there).
Inputs lie among NaN (row ends, what surrounds a buffer), outputs among
values that must not change.
"""
import pytest
import torch

import layers_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
INPUT = {"f32": 0, "bf16": 1, "f16": 2}
CANARY = 77.0


@pytest.fixture(scope="module")
def lib():
    from dense_gemm_optimisation_amd import binding
    binding.library()
    return binding


class Matrix:
    """rows x cols in the middle of a larger buffer, `pad` elements behind each row, `lead` before the first."""

    def __init__(self, value, kind, pad=0, lead=0, fill=float("nan")):
        batch = value.shape[:-2]
        self.rows, self.cols = value.shape[-2:]
        self.kind, self.ld, self.lead = kind, self.cols + pad, lead
        n = 1
        for b in batch:
            n *= b
        self.stride = self.rows * self.ld + 8
        self.buffer = torch.full((lead + n * self.stride + 64,), fill, dtype=ref.TORCH[kind], device=DEV)
        self.view = self.buffer[lead:].as_strided((n, self.rows, self.cols), (self.stride, self.ld, 1))
        self.view.copy_(value.reshape(n, self.rows, self.cols))
        if not batch:
            self.view = self.view[0]
        self.before = self.buffer.clone()

    @property
    def ptr(self):
        return self.buffer.data_ptr() + self.lead * self.buffer.element_size()

    def get(self):
        return self.view.cpu().double()

    def untouched(self, whole=False):
        """Nothing outside the matrix changed (nothing at all, if `whole`)."""
        now, before = self.buffer.clone(), self.before.clone()
        if not whole:
            for b in (now, before):
                v = b[self.lead:].as_strided(self.view.shape, self.view.stride())
                v.fill_(0)
        return torch.equal(now.nan_to_num(nan=1e4), before.nan_to_num(nan=1e4))


def draw(shape, kind, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(*shape, generator=g, dtype=torch.float64)).to(ref.TORCH[kind])


def close(got, want, bound, what):
    off = (got - want).abs()
    bad = ~(off <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {(off / bound).max().item():.3g} of the bound"


def space(n):
    return torch.full((max(n, 16) // 4 + 4,), float("nan"), device=DEV)


# ---------------------------------------------------------------- gemm_linear and its gradient
def weights(b, order, kind, pad, lead):
    """B (K x N) as stored."""
    return Matrix(b.t() if order == "nk" else b, kind, pad, lead)


def run_linear(lib, M, N, K, kind="bf16", order="nk", act="gelu", bias=True, beta=0.0, keep=False, out=None, alpha=1.0, pad=8,
               lead=0, in_place=False, workspace=True, seed=0, expect=None, compare=True):
    out = out or kind
    a, b = draw((M, K), kind, seed), draw((K, N), kind, seed + 1, K ** -0.5 if K else 1.0)
    bi = draw((N,), kind, seed + 2) if bias else None
    r = draw((M, N), out, seed + 3)
    ma, mb = Matrix(a, kind, pad, lead), weights(b, order, kind, pad, lead)
    mbias = Matrix(bi[None], kind, 0, lead) if bias else None
    mr = Matrix(r, out, pad, lead) if not in_place else None
    mc = Matrix(r if in_place else torch.full((M, N), CANARY), out, pad, lead, CANARY)
    mz = Matrix(torch.full((M, N), CANARY), kind, pad, lead, CANARY) if keep else None
    ws = space(lib.linear_workspace_size(M, N, K)) if workspace else None
    res = mc if in_place else mr
    args = (M, N, K, alpha, ma.ptr, ma.ld, mb.ptr, mb.ld, lib.COL_MAJOR if order == "nk" else lib.ROW_MAJOR, INPUT[kind],
            mbias.ptr if bias else 0, {"none": 0, "relu": 1, "gelu": 2, "silu": 3}[act], beta, res.ptr if beta else 0, res.ld,
            mc.ptr, mc.ld, INPUT[out], mz.ptr if keep else 0, mz.ld if keep else 0, ws.data_ptr() if workspace else 0,
            ws.numel() * 4 if workspace else 0)
    name = lib.linear_kernel_name(*args)
    if expect:
        assert name == expect
    print(name, M, N, K, kind, order, act, flush=True)
    lib.gemm_linear(*args)
    torch.cuda.synchronize()
    if compare:
        want, bound = ref.linear(a, b, bi, alpha, act, beta, r, out, kind)
        close(mc.get(), want["out"], bound["out"], f"C of {name}")
        if keep:
            close(mz.get(), want["z"], bound["z"], f"Z of {name}")
    assert mc.untouched() and ma.untouched(True) and mb.untouched(True)
    assert mz is None or mz.untouched()
    return mc, args


SHAPES = [(1, 1, 1), (1, 64, 64), (3, 17, 5), (16, 48, 136), (16, 1000, 520), (17, 130, 72), (33, 7, 300), (127, 129, 64), (128, 256, 128),
          (129, 127, 65), (250, 1000, 515), (64, 264, 2048)]


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("order", ["nk", "kn"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear_shapes(lib, M, N, K, order, kind):
    run_linear(lib, M, N, K, kind, order, act="gelu", beta=0.75, keep=True)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("M,N,K,pad,lead", [(16, 80, 256, 8, 8), (40, 136, 264, 0, 0), (130, 140, 70, 3, 1)])
@pytest.mark.parametrize("bias,beta,keep,out", [(False, 0.0, False, None), (True, 0.0, True, "f32"), (False, -1.5, False, "f32"),
                                                (True, 1.0, False, None)])
def test_linear_epilogue(lib, M, N, K, pad, lead, act, bias, beta, keep, out):
    run_linear(lib, M, N, K, act=act, bias=bias, beta=beta, keep=keep, out=out, pad=pad, lead=lead, alpha=1.25)


@pytest.mark.parametrize("kernel,M,N,K,order,pad,workspace", [
    ("linear_few_16", 16, 400, 1304, "nk", 8, True), ("linear_few_16", 5, 33, 24, "nk", 8, False),
    ("linear_mfma_128", 100, 200, 1000, "nk", 8, False), ("linear_mfma_128", 130, 200, 192, "kn", 8, True),
    ("linear_mfma_128_split", 40, 300, 1000, "nk", 8, True), ("linear_mfma_128_split", 8, 520, 4160, "kn", 8, True),
    ("linear_mfma_any", 100, 200, 1001, "nk", 1, False), ("linear_mfma_any", 100, 203, 96, "kn", 5, True),
    ("linear_mfma_any_split", 9, 203, 1001, "nk", 3, True), ("linear_mfma_any_split", 300, 77, 999, "kn", 3, True),
])
@pytest.mark.parametrize("backward", [False, True])
def test_linear_kernels(lib, kernel, M, N, K, order, pad, workspace, backward):
    if backward:
        run_backward(lib, M, N, K, order=order, pad=pad, workspace=workspace, bias=workspace, expect=kernel)
    else:
        run_linear(lib, M, N, K, order=order, pad=pad, workspace=workspace, beta=1.0, keep=True, expect=kernel)


@pytest.mark.parametrize("kind,order", [("bf16", "nk"), ("f16", "kn")])
@pytest.mark.parametrize("backward", [False, True])
def test_linear_large_tiles(lib, kind, order, backward):
    """Enough tiles of 256 x 256, ragged in every dimension."""
    M, N, K = 3600, 3656, 72
    if backward:
        run_backward(lib, M, N, K, kind, order, expect="linear_mfma_256")
    else:
        run_linear(lib, M, N, K, kind, order, beta=1.0, keep=True, expect="linear_mfma_256")


@pytest.mark.parametrize("kernel,M,N,K,kind,order,pad,lead", [
    ("linear_packed", 1030, 1100, 515, "f16", "nk", 1, 1), ("linear_packed", 1100, 1025, 600, "bf16", "kn", 3, 0),
    ("linear_packed", 1024, 1024, 1024, "bf16", "nk", 8, 3), ("linear_packed", 1030, 17001, 520, "f16", "kn", 7, 0),
    ("linear_mfma_256_rounds", 300, 33030, 520, "bf16", "nk", 8, 0), ("linear_mfma_256_rounds", 2300, 8000, 576, "f16", "kn", 0, 0),
])
@pytest.mark.parametrize("backward", [False, True])
def test_linear_copies_and_rounds(lib, kernel, M, N, K, kind, order, pad, lead, backward):
    """Operands copied for direct loads; tiles that whole rounds leave over."""
    expect = kernel
    if (M, N, K) == (1024, 1024, 1024):
        expect = "linear_mfma_any_split"  # the workspace has no room for copies of rows of whole chunks
    if backward:
        run_backward(lib, M, N, K, kind, order, pad=pad, lead=lead, expect=expect)
    else:
        run_linear(lib, M, N, K, kind, order, beta=1.0, keep=True, pad=pad, lead=lead, expect=expect)


@pytest.mark.parametrize("M,N,K", [(16, 64, 256), (70, 136, 128), (130, 140, 71)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_linear_in_place(lib, M, N, K, out):
    run_linear(lib, M, N, K, beta=1.0, in_place=True, out=out)


@pytest.mark.parametrize("M,N", [(1, 1), (20, 37), (130, 264)])
def test_linear_without_product(lib, M, N):
    """K = 0 and alpha = 0: neither A nor B is read."""
    run_linear(lib, M, N, 0, beta=1.0, keep=True)
    bi, c = draw((N,), "bf16", 4), Matrix(torch.full((M, N), CANARY), "bf16", 3, 0, CANARY)
    b = bi.to(DEV)
    lib.gemm_linear(M, N, 50, 0.0, 0, 50, 0, 50, 1, 1, b.data_ptr(), 3, 0.0, 0, 0, c.ptr, c.ld, 1)
    torch.cuda.synchronize()
    want, bound = ref.linear(torch.zeros(M, 1), torch.zeros(1, N), bi, 0.0, "silu", 0, None, "bf16", "bf16")
    close(c.get(), want["out"], bound["out"], "alpha = 0")
    assert c.untouched()


@pytest.mark.parametrize("M,N,K", [(16, 64, 256), (130, 136, 128), (40, 64, 1024), (30, 75, 99)])
def test_linear_unusual_values(lib, M, N, K):
    """Infinities and NaN stay in the rows and columns they belong to; a residual that beta leaves out is not read."""
    a, b = draw((M, K), "bf16", 1), draw((N, K), "bf16", 2)
    a[3, 5], b[7, 2] = float("inf"), float("nan")
    da, db = a.to(DEV), b.to(DEV)
    r = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    c = torch.zeros(M, N, dtype=torch.bfloat16, device=DEV)
    ws = space(lib.linear_workspace_size(M, N, K))
    lib.gemm_linear(M, N, K, 1.0, da.data_ptr(), K, db.data_ptr(), K, 1, 1, 0, 0, 0.0, r.data_ptr(), N, c.data_ptr(), N, 1, 0, 0,
                    ws.data_ptr(), ws.numel() * 4)
    torch.cuda.synchronize()
    got, want = c.cpu(), a.double() @ b.double().t()
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.isinf(), want.isinf())
    assert got[:, 7].isnan().all() and not got[4:, :7].isnan().any()


def test_linear_many_tiles(lib):
    """More tiles than one launch takes."""
    M = (1 << 22) * 128 + 700
    a = torch.randint(-8, 9, (M,), dtype=torch.int8, device=DEV, generator=torch.Generator(device=DEV).manual_seed(6)).bfloat16()
    b, c = torch.full((1,), 3.0, dtype=torch.bfloat16, device=DEV), torch.full((M,), 7.0, dtype=torch.bfloat16, device=DEV)
    lib.gemm_linear(M, 1, 1, 1.0, a.data_ptr(), 1, b.data_ptr(), 1, 1, 1, 0, 0, 0.0, 0, 1, c.data_ptr(), 1, 1)
    torch.cuda.synchronize()
    assert torch.equal(c, 3 * a)


def run_backward(lib, M, N, K, kind="bf16", order="nk", act="gelu", beta=0.0, out=None, alpha=1.0, pad=8, lead=0, in_place=False,
                 workspace=True, bias=True, seed=0, expect=None):
    out = out or kind
    a, b = draw((M, K), kind, seed), draw((K, N), kind, seed + 1, K ** -0.5 if K else 1.0)
    z, db = draw((M, N), kind, seed + 2, 1.5), draw((N,), "f32", seed + 3)
    ma, mb = Matrix(a, kind, pad, lead), weights(b, order, kind, pad, lead)
    mz = Matrix(z, kind, pad, lead)
    md = mz if in_place else Matrix(torch.full((M, N), CANARY), out, pad, lead, CANARY)
    mdb = Matrix(db[None], "f32", 0, 3, CANARY)
    ws = space(lib.linear_workspace_size(M, N, K)) if workspace else None
    args = (M, N, K, alpha, ma.ptr, ma.ld, mb.ptr, mb.ld, lib.COL_MAJOR if order == "nk" else lib.ROW_MAJOR, INPUT[kind], mz.ptr,
            mz.ld, {"none": 0, "relu": 1, "gelu": 2, "silu": 3}[act], md.ptr, md.ld, INPUT[out], beta, mdb.ptr if bias else 0,
            ws.data_ptr() if workspace else 0, ws.numel() * 4 if workspace else 0)
    name = lib.linear_backward_kernel_name(*args)
    if expect:
        assert name == expect
    print(name, M, N, K, kind, order, act, flush=True)
    lib.gemm_linear_backward(*args)
    torch.cuda.synchronize()
    want, bound = ref.through(*ref.product(a, b, alpha), z, act, db, beta, out)
    close(md.get(), want["out"], bound["out"], f"D of {name}")
    if bias:
        close(mdb.get()[0], want["d_bias"], bound["d_bias"], f"dbias of {name}")
    assert md.untouched() and mdb.untouched(not bias)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("order", ["nk", "kn"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear_backward_shapes(lib, M, N, K, order, kind):
    run_backward(lib, M, N, K, kind, order, beta=1.0)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("M,N,K,pad,lead", [(16, 80, 256, 8, 8), (40, 136, 264, 0, 0), (130, 140, 70, 3, 1)])
@pytest.mark.parametrize("beta,out,in_place,bias", [(0.0, "f32", False, True), (-0.5, None, False, True), (0.0, None, True, True),
                                                    (0.0, None, False, False)])
def test_linear_backward_epilogue(lib, M, N, K, pad, lead, act, beta, out, in_place, bias):
    run_backward(lib, M, N, K, act=act, beta=beta, out=out, pad=pad, lead=lead, alpha=-0.75, in_place=in_place, bias=bias)


def test_linear_backward_no_rows(lib):
    """No rows: the bias's gradient is what beta leaves."""
    d = torch.arange(70, dtype=torch.float32, device=DEV)
    lib.gemm_linear_backward(0, 70, 8, 1.0, 0, 8, 0, 8, 1, 1, 0, 70, 2, 0, 70, 1, 0.5, d.data_ptr())
    lib.gemm_activation_backward(0, 70, 0, 70, 1, 0, 70, 1, 2, 0, 70, 1, 0.5, d.data_ptr())
    torch.cuda.synchronize()
    assert torch.equal(d.cpu(), torch.arange(70, dtype=torch.float32) / 4)
    lib.gemm_linear_backward(0, 70, 8, 1.0, 0, 8, 0, 8, 1, 1, 0, 70, 2, 0, 70, 1, 0.0, d.data_ptr())
    torch.cuda.synchronize()
    assert not d.any()


def test_linear_backward_is_the_gradient(lib):
    """D and dbias against differences of the forward call's own outputs in fp32."""
    M, N, K = 24, 40, 64
    x, w, bi = draw((M, K), "f16", 1), draw((N, K), "f16", 2, K ** -0.5), draw((N,), "f16", 3)
    up = draw((M, 32), "f16", 4)
    w2 = draw((32, N), "f16", 5, N ** -0.5)
    d = lambda t: t.to(DEV)  # noqa: E731
    dx, dw, dup, dw2 = d(x), d(w), d(up), d(w2)
    ws = space(lib.linear_workspace_size(M, N, K))

    def forward(b):
        c = torch.zeros(M, N, device=DEV)
        z = torch.zeros(M, N, dtype=torch.float16, device=DEV)
        db = d(b)
        lib.gemm_linear(M, N, K, 1.0, dx.data_ptr(), K, dw.data_ptr(), K, 1, 2, db.data_ptr(), 2, 0.0, 0, 0, c.data_ptr(), N, 0,
                        z.data_ptr(), N, ws.data_ptr(), ws.numel() * 4)
        torch.cuda.synchronize()
        return c.cpu().double(), z
    _, z = forward(bi)
    g = torch.zeros(M, N, device=DEV)
    gb = torch.zeros(N, device=DEV)
    lib.gemm_linear_backward(M, N, 32, 1.0, dup.data_ptr(), 32, dw2.data_ptr(), N, 0, 2, z.data_ptr(), N, 2, g.data_ptr(), N, 0, 0.0,
                             gb.data_ptr(), ws.data_ptr(), ws.numel() * 4)
    torch.cuda.synchronize()
    flow = up.double() @ w2.double()
    # a step of 2^-4 in the bias, exact in fp16 for |bias| < 2^6 up to its own rounding, which the difference divides by
    hi, lo = (bi + 2.0 ** -4).half(), (bi - 2.0 ** -4).half()
    step = (hi.double() - lo.double())
    diff = ((forward(hi)[0] - forward(lo)[0]) * flow / step).sum(0)
    # GELU's third derivative is below 1.7 in magnitude: step^2 / 6 of it; z is kept in fp16 (2^-11 |z|, |z| < 8, slope's
    # derivative below 0.8); fp32 sums
    bound = (flow.abs() * (1.7 * (2.0 ** -4) ** 2 / 6 + 0.8 * 8 * 2.0 ** -11 + 2.0 ** -10)).sum(0)
    assert ((gb.cpu().double() - diff).abs() <= bound).all()


# ---------------------------------------------------------------- gemm_activation_backward
def run_activation(lib, M, N, kinds, act, beta=0.0, in_place=None, want_d=True, bias=True, pad=3, lead=1):
    ka, kz, kd = kinds
    a, z, db = draw((M, N), ka, 1), draw((M, N), kz, 2, 1.5), draw((N,), "f32", 3)
    ma, mz = Matrix(a, ka, pad, lead), Matrix(z, kz, pad, lead)
    md = {"a": ma, "z": mz, None: Matrix(torch.full((M, N), CANARY), kd, pad, lead, CANARY)}[in_place]
    mdb = Matrix(db[None], "f32", 0, 3, CANARY)
    ws = space(lib.activation_backward_workspace_size(M, N))
    print(M, N, kinds, act, flush=True)
    lib.gemm_activation_backward(M, N, ma.ptr, ma.ld, INPUT[ka], mz.ptr, mz.ld, INPUT[kz],
                                 {"none": 0, "relu": 1, "gelu": 2, "silu": 3}[act], md.ptr if want_d else 0, md.ld, INPUT[md.kind],
                                 beta, mdb.ptr if bias else 0, ws.data_ptr() if bias else 0, ws.numel() * 4 if bias else 0)
    torch.cuda.synchronize()
    want, bound = ref.through(a.double(), torch.zeros(M, N, dtype=torch.float64), z, act, db, beta, md.kind)
    if want_d:
        close(md.get(), want["out"], bound["out"], "D")
    if bias:
        close(mdb.get()[0], want["d_bias"], bound["d_bias"], "dbias")
    assert md.untouched(not want_d and in_place is None) and mdb.untouched(not bias)


@pytest.mark.parametrize("kinds", [(a, z, d) for a in INPUT for z in INPUT for d in INPUT])
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_activation_backward_types(lib, kinds, act):
    run_activation(lib, 70, 100, kinds, act, beta=1.0)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("M,N,pad,lead", [(1, 1, 0, 0), (1, 4097, 0, 0), (129, 63, 1, 1), (128, 64, 0, 0), (1000, 9, 7, 0), (257, 520, 8, 8)])
def test_activation_backward_shapes(lib, M, N, pad, lead, act):
    run_activation(lib, M, N, ("bf16", "bf16", "bf16"), act, pad=pad, lead=lead)


@pytest.mark.parametrize("in_place,want_d,bias", [("a", True, True), ("z", True, True), (None, False, True), (None, True, False)])
def test_activation_backward_forms(lib, in_place, want_d, bias):
    run_activation(lib, 100, 70, ("f16", "f16", "f16"), "silu", beta=0.25, in_place=in_place, want_d=want_d, bias=bias)


def test_activation_backward_many_rows(lib):
    """More rows than a grid has rows of workgroups of 128; whole numbers, so every sum is exact."""
    M, N = 65535 * 128 + 300, 8
    g = torch.Generator(device=DEV).manual_seed(5)
    a = torch.randint(-1, 2, (M, N), device=DEV, generator=g).bfloat16()
    z = torch.randint(-1, 2, (M, N), device=DEV, generator=g).bfloat16()
    d, db = torch.empty_like(a), torch.zeros(N, device=DEV)
    ws = space(lib.activation_backward_workspace_size(M, N))
    lib.gemm_activation_backward(M, N, a.data_ptr(), N, 1, z.data_ptr(), N, 1, 1, d.data_ptr(), N, 1, 0.0, db.data_ptr(),
                                 ws.data_ptr(), ws.numel() * 4)
    want = torch.where(z > 0, a, torch.zeros_like(a))
    assert torch.equal(d, want)
    assert torch.equal(db, want.float().sum(0, dtype=torch.float64).float())


# ---------------------------------------------------------------- gemm_experts_layer
def experts_case(lib, T, E, k, D, H, kind="bf16", form="same", act="silu", beta=0.0, out=None, seed=0, ids=None, pad=8):
    out = out or kind
    g = torch.Generator().manual_seed(seed)
    x = draw((T, D), kind, seed + 1)
    if ids is None:
        ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int()
    gates = torch.rand(T, k, generator=g)
    values, stored = [], []
    for rows, K, i in ((2 * H, D, 2), (D, H, 3)):
        if form == "same":
            w = draw((E, rows, K), kind, seed + i, 0.5 * K ** -0.5)
            width = -(-K // 8) * 8 + pad
            m = torch.full((E, rows, width), float("nan"), dtype=ref.TORCH[kind])
            m[:, :, :K] = w
            values.append([v.double() for v in w])
            stored.append((m.to(DEV), None))
        else:
            f8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}[form]
            codes = (8 * torch.randn(E, rows, K, generator=g)).to(f8)
            kb, rb = -(-K // 128), -(-rows // 128)
            scale = 0.125 * K ** -0.5 * torch.exp(0.5 * torch.randn(E, kb, rb, generator=g)) / 2
            width = -(-K // 16) * 16 + 16
            m = torch.full((E, rows, width), 0x7F, dtype=torch.uint8)
            m[:, :, :K] = codes.view(torch.uint8)
            sm = torch.full((E, kb, rb + 1), float("nan"))
            sm[:, :, :rb] = scale
            s = scale.double().transpose(1, 2).repeat_interleave(128, 1)[:, :rows].repeat_interleave(128, 2)[:, :, :K]
            values.append(list(codes.double() * s))
            stored.append((m.to(DEV), sm.to(DEV)))
    mx = Matrix(x, kind, -D % 8 + 8)
    before = draw((T, D), out, seed + 9)
    my = Matrix(before, out, 3, 1, CANARY)
    return dict(T=T, E=E, k=k, D=D, H=H, kind=kind, form=form, act=act, beta=beta, out=out, x=x, ids=ids, gates=gates, values=values,
                stored=stored, mx=mx, my=my, before=before, dids=ids.to(DEV), dgates=gates.to(DEV),
                ws=space(lib.experts_layer_workspace_size(T, E, k, D, H)))


def experts_call(lib, c, **kw):
    (up, su), (down, sd) = c["stored"]

    def operand(w, s):
        return (w.data_ptr(), w.stride(1), w.stride(0)) + ((0, 0, 0) if s is None else (s.data_ptr(), s.stride(1), s.stride(0)))
    form = {"same": 0, "e4m3": 1, "e5m2": 2}[c["form"]]
    lib.gemm_experts_layer(c["T"], c["E"], c["k"], c["D"], c["H"], c["mx"].ptr, c["mx"].ld, INPUT[c["kind"]], c["dids"].data_ptr(),
                           c["dgates"].data_ptr(), form, *operand(up, su), *operand(down, sd), {"relu": 1, "gelu": 2, "silu": 3}[c["act"]],
                           c["beta"], c["my"].ptr, c["my"].ld, INPUT[c["out"]], c["ws"].data_ptr(), c["ws"].numel() * 4, **kw)


def experts_check(lib, *args, **kw):
    c = experts_case(lib, *args, **kw)
    print(args, kw, flush=True)
    experts_call(lib, c)
    torch.cuda.synchronize()
    want, bound = ref.experts_layer(c["x"], c["ids"], c["gates"], *c["values"], c["act"], c["beta"], c["before"], c["out"], c["kind"])
    close(c["my"].get(), want, bound, "Y")
    assert c["my"].untouched() and c["mx"].untouched(True)


@pytest.mark.parametrize("form", ["same", "e4m3", "e5m2"])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("T,E,k,D,H", [(1, 1, 1, 1, 1), (1, 8, 2, 64, 48), (1, 64, 8, 1032, 264), (5, 4, 4, 130, 77), (16, 33, 3, 200, 129),
                                       (17, 8, 2, 72, 140), (33, 60, 6, 136, 136), (64, 3, 2, 264, 33)])
def test_experts_layer_shapes(lib, T, E, k, D, H, kind, form):
    experts_check(lib, T, E, k, D, H, kind, form)


@pytest.mark.parametrize("act", ["relu", "gelu", "silu"])
@pytest.mark.parametrize("beta,out", [(0.0, "f32"), (1.0, None), (-0.5, "f32")])
def test_experts_layer_epilogue(lib, act, beta, out):
    experts_check(lib, 9, 6, 2, 136, 72, act=act, beta=beta, out=out)


def test_experts_layer_ids(lib):
    """Ids outside the experts take no part, whatever their weights; one that a token holds twice counts twice; a token
    without experts keeps beta * Y; every token may choose one expert."""
    ids = torch.tensor([[-1, -1], [3, 3], [0, -1], [7, 1], [-5, 2], [1 << 30, 1], [5, 0]], dtype=torch.int32)
    for beta in (0.0, 1.0):
        c = experts_case(lib, 7, 7, 2, 72, 40, ids=ids, beta=beta)
        c["gates"][0] = float("nan")
        c["dgates"].copy_(c["gates"])
        experts_call(lib, c)
        torch.cuda.synchronize()
        want, bound = ref.experts_layer(c["x"], ids, c["gates"], *c["values"], "silu", beta, c["before"], "bf16", "bf16")
        close(c["my"].get(), want, bound, "Y")
    one = torch.full((64, 1), 2, dtype=torch.int32)
    experts_check(lib, 64, 5, 1, 136, 72, ids=one)
    experts_check(lib, 40, 5, 1, 136, 72, ids=torch.full((40, 1), -1, dtype=torch.int32), beta=1.0)


def test_experts_layer_limits(lib):
    """As many experts and choices as the call takes."""
    experts_check(lib, 64, 1024, 32, 16, 8)


# ---------------------------------------------------------------- gemm_orthogonalize
def matrix(M, N, seed, spectrum):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, N, generator=g, dtype=torch.float64)
    if spectrum == "few":  # a few directions hold most of the norm
        r = max(1, min(M, N) // 16)
        x = 0.3 * x + torch.randn(M, r, generator=g, dtype=torch.float64) @ torch.randn(r, N, generator=g, dtype=torch.float64)
    return x


def run_ortho(lib, M, N, kind="f32", out="f32", steps=5, coefficients=None, eps=1e-7, alpha=1.0, beta=0.0, batch=1, scale=1e-3, pad=3,
              lead=1, spectrum="plain", seed=0):
    x = torch.stack([scale * matrix(M, N, seed + b, spectrum) for b in range(batch)]).to(ref.TORCH[kind])
    o = draw((batch, M, N), out, seed + 50, 0.5)
    mg, mo = Matrix(x, kind, pad, lead), Matrix(o, out, pad, lead, CANARY)
    ws = space(lib.orthogonalize_workspace_size(M, N, batch))
    print(lib.orthogonalize_kernel_name(M, N, batch), M, N, kind, out, batch, flush=True)
    lib.gemm_orthogonalize(M, N, mg.ptr, mg.ld, INPUT[kind], steps, coefficients, eps, alpha, beta, mo.ptr, mo.ld, INPUT[out],
                           ws.data_ptr(), ws.numel() * 4, batch=batch, stride_g=mg.stride, stride_o=mo.stride)
    torch.cuda.synchronize()
    assert mo.untouched() and mg.untouched(True)
    got = mo.get()
    for b in range(batch):
        want = ref.newton_schulz(x[b], steps, coefficients, eps)
        drift = torch.linalg.matrix_norm(ref.newton_schulz(x[b], steps, coefficients, eps, rounding=True) - want).item()
        size = torch.linalg.matrix_norm(want).item()
        y = alpha * want + (beta * o[b].double() if beta else 0.0)
        # twice the same roundings' drift (their signs differ: sums in fp32 are in another order), fp32's, the output's
        bound = abs(alpha) * (2 * drift + 2.0 ** -16 * size) + ref.HALF[out] * torch.linalg.matrix_norm(y).item() + 1e-30
        off = torch.linalg.matrix_norm(got[b] - y).item()
        assert off <= bound, f"{M}x{N} [{b}]: off {off:.3g} of {bound:.3g}"
    return got


@pytest.mark.parametrize("spectrum", ["plain", "few"])
@pytest.mark.parametrize("M,N", [(1, 1), (1, 300), (300, 1), (2, 2), (7, 5), (64, 64), (128, 128), (33, 200), (129, 77), (130, 260), (257, 256),
                                 (500, 137)])
def test_orthogonalize_shapes(lib, M, N, spectrum):
    run_ortho(lib, M, N, spectrum=spectrum)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,N", [(40, 70), (200, 96)])
def test_orthogonalize_types(lib, kind, out, M, N):
    run_ortho(lib, M, N, kind, out, alpha=-0.02, beta=0.99)


@pytest.mark.parametrize("M,N,batch", [(64, 64, 5), (128, 40, 3), (150, 200, 4)])
def test_orthogonalize_batches(lib, M, N, batch):
    run_ortho(lib, M, N, batch=batch, beta=1.0)


@pytest.mark.parametrize("M,N,batch", [(190, 200, 200), (250, 250, 128), (250, 130, 128), (260, 250, 60), (250, 260, 250)])
def test_orthogonalize_every_tile(lib, M, N, batch):
    """The symmetric products' tiles of 192, 128 in two rounds and in one, and 256."""
    run_ortho(lib, M, N, batch=batch, steps=3)


def test_orthogonalize_large(lib):
    """Enough tiles of 256 x 256 for the large kernel, ragged."""
    assert lib.orthogonalize_kernel_name(3600, 3590, 1) == "orthogonalize_mfma_256"
    run_ortho(lib, 3600, 3590, "bf16", "bf16", steps=2)


def test_orthogonalize_coefficients(lib):
    """Each step its own; the cubic steps bring every singular value to 1."""
    steps = [(4.0848, -6.8946, 2.9270), (3.9505, -6.3029, 2.6377), (3.7418, -5.5913, 2.3037), (2.8769, -3.1427, 1.2046),
             (2.8366, -3.0525, 1.2012), (1.5, -0.5, 0.0), (1.5, -0.5, 0.0), (1.5, -0.5, 0.0)]
    x = run_ortho(lib, 96, 160, steps=8, coefficients=steps)[0]
    # the singular values end at 1; the roundings leave a few 2^-11 of the elements' root mean square
    s = torch.linalg.svdvals(x)
    assert (s - 1).abs().max() < 0.02


@pytest.mark.parametrize("scale", [1e-30, 1e-12, 1.0, 1e15, 1e30])
def test_orthogonalize_scales(lib, scale):
    """The norm's square leaves fp32's range; eps = 0."""
    run_ortho(lib, 60, 90, scale=scale, eps=0.0)


@pytest.mark.parametrize("M,N", [(70, 60), (60, 70)])
def test_orthogonalize_unusual_values(lib, M, N):
    """A matrix of zeros gives beta * O, one with an infinity or a NaN NaN throughout, and the others of the batch are not touched
    by it; eps bounds the norm."""
    x = torch.stack([0 * matrix(M, N, 1, "plain"), matrix(M, N, 2, "plain"), matrix(M, N, 3, "plain"), matrix(M, N, 4, "plain")]).float()
    x[1, 5, 6], x[2, 3, 3] = float("inf"), float("nan")
    d, o = x.to(DEV), torch.ones(4, M, N, device=DEV)
    ws = space(lib.orthogonalize_workspace_size(M, N, 4))
    for eps in (0.0, 1e-7):
        o.fill_(1)
        lib.gemm_orthogonalize(M, N, d.data_ptr(), N, 0, 5, None, eps, 1.0, 0.5, o.data_ptr(), N, 0, ws.data_ptr(), ws.numel() * 4,
                               batch=4, stride_g=M * N, stride_o=M * N)
        torch.cuda.synchronize()
        assert (o[0] == 0.5).all() and o[1].isnan().all() and o[2].isnan().all()
        off = torch.linalg.matrix_norm(o[3].cpu().double() - 0.5 - ref.newton_schulz(x[3], 5)).item()
        assert off <= 2.0 ** -7 * min(M, N) ** 0.5
    run_ortho(lib, M, N, eps=1e3)


# ---------------------------------------------------------------- together
class Layer:
    """A feed-forward layer's training step: forward, backward, and its first weight's update, as a program holds it."""

    def __init__(self, lib, T, D, H, seed):
        t = torch.bfloat16
        new = lambda *s, dtype=t: torch.zeros(*s, dtype=dtype, device=DEV)  # noqa: E731
        self.lib, self.T, self.D, self.H = lib, T, D, H
        self.x, self.g = (draw((T, D), "bf16", seed + i).to(DEV) for i in (0, 1))
        self.w1, self.w2 = draw((H, D), "bf16", seed + 2, D ** -0.5).to(DEV), draw((D, H), "bf16", seed + 3, H ** -0.5).to(DEV)
        self.b1, self.b2 = draw((H,), "bf16", seed + 4).to(DEV), draw((D,), "bf16", seed + 5).to(DEV)
        self.z, self.h, self.dz = new(T, H), new(T, H), new(T, H)
        self.y, self.dx, self.dw1 = new(T, D), new(T, D), new(H, D, dtype=torch.float32)
        self.db1, self.db2 = new(H, dtype=torch.float32), new(D, dtype=torch.float32)
        self.step = new(H, D, dtype=torch.float32)
        n = max(lib.linear_workspace_size(T, H, D), lib.linear_workspace_size(T, D, H), lib.activation_backward_workspace_size(T, D),
                lib.orthogonalize_workspace_size(H, D))
        self.ws = space(n)

    def run(self, stream=None):
        lib, T, D, H = self.lib, self.T, self.D, self.H
        p = lambda t: t.data_ptr()  # noqa: E731
        ws = dict(workspace=p(self.ws), workspace_bytes=self.ws.numel() * 4)
        s = dict(stream=stream)
        lib.gemm_linear(T, H, D, 1.0, p(self.x), D, p(self.w1), D, lib.COL_MAJOR, lib.INPUT_BF16, p(self.b1), lib.ACT_GELU, 0.0, 0, 0,
                        p(self.h), H, lib.OUTPUT_BF16, p(self.z), H, **ws, **s)
        lib.gemm_linear(T, D, H, 1.0, p(self.h), H, p(self.w2), H, lib.COL_MAJOR, lib.INPUT_BF16, p(self.b2), lib.ACT_NONE, 1.0,
                        p(self.x), D, p(self.y), D, lib.OUTPUT_BF16, **ws, **s)
        lib.gemm_activation_backward(T, D, p(self.g), D, lib.INPUT_BF16, 0, 0, lib.INPUT_BF16, lib.ACT_NONE, 0, 0, lib.OUTPUT_F32, 0.0,
                                     p(self.db2), **ws, **s)
        lib.gemm_linear_backward(T, H, D, 1.0, p(self.g), D, p(self.w2), H, lib.ROW_MAJOR, lib.INPUT_BF16, p(self.z), H, lib.ACT_GELU,
                                 p(self.dz), H, lib.OUTPUT_BF16, 0.0, p(self.db1), **ws, **s)
        # the input's gradient takes the residual's too; the weight's gradient is the library's plain product
        lib.gemm_linear(T, D, H, 1.0, p(self.dz), H, p(self.w1), D, lib.ROW_MAJOR, lib.INPUT_BF16, 0, lib.ACT_NONE, 1.0, p(self.g), D,
                        p(self.dx), D, lib.OUTPUT_BF16, **ws, **s)
        lib.gemm_bf16(H, D, T, 1.0, p(self.dz), H, lib.COL_MAJOR, p(self.x), D, lib.ROW_MAJOR, 0.0, p(self.dw1), D, lib.ROW_MAJOR,
                      lib.DTYPE_F32, **s)
        lib.gemm_orthogonalize(H, D, p(self.dw1), D, lib.INPUT_F32, 5, None, 1e-7, -0.02, 1.0, p(self.step), D, lib.OUTPUT_F32,
                               p(self.ws), self.ws.numel() * 4, **s)

    def outputs(self):
        return [t.clone() for t in (self.z, self.h, self.y, self.db2, self.dz, self.db1, self.dx, self.dw1, self.step)]

    def clear(self):
        for t in (self.z, self.h, self.y, self.db2, self.dz, self.db1, self.dx, self.dw1, self.step):
            t.zero_()


@pytest.mark.parametrize("T,D,H", [(40, 72, 200), (256, 128, 512)])
def test_training_step(lib, T, D, H):
    layer = Layer(lib, T, D, H, 1)
    layer.run()
    torch.cuda.synchronize()
    z, h, y, db2, dz, db1, dx, dw1, step = (t.cpu().double() for t in layer.outputs())
    x, g, w1, w2, b1, b2 = (t.cpu().double() for t in (layer.x, layer.g, layer.w1, layer.w2, layer.b1, layer.b2))
    x, w1, b1, w2 = (t.requires_grad_() for t in (x, w1, b1, w2))
    pre = x @ w1.t() + b1
    out = x + torch.nn.functional.gelu(pre) @ w2.t() + b2
    out.backward(g)
    # every stored activation is rounded to bf16 once: 2^-8 of the largest of a sum's terms, sums of up to H of them random in sign
    # (root mean square), with a margin of 4 over 3 such roundings
    for got, want in ((z, pre.detach()), (y, out.detach()), (dx, x.grad), (db1, b1.grad), (dw1, w1.grad), (db2, g.sum(0))):
        off = torch.linalg.vector_norm(got - want) / torch.linalg.vector_norm(want)
        assert off < 3 * 4 * 2.0 ** -8, off
    want = -0.02 * ref.newton_schulz(dw1, 5, eps=1e-7)
    drift = torch.linalg.matrix_norm(want + 0.02 * ref.newton_schulz(dw1, 5, eps=1e-7, rounding=True))
    assert torch.linalg.matrix_norm(step - want) <= 2 * drift + 2.0 ** -16 * torch.linalg.matrix_norm(want)


def test_training_step_captured_and_on_streams(lib):
    """Replays of a graph, and two layers at once on two streams, give what the eager calls gave, bit for bit."""
    a, b = Layer(lib, 40, 72, 200, 1), Layer(lib, 130, 264, 136, 2)
    for layer in (a, b):
        layer.run()
    torch.cuda.synchronize()
    want = a.outputs(), b.outputs()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        a.run()
    for i in range(3):
        a.clear()
        noise = torch.randn(512, 512, device=DEV) @ torch.randn(512, 512, device=DEV)
        graph.replay()
        assert noise.isfinite().all()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(a.outputs(), want[0])), f"replay {i}"
    for i in range(3):
        a.clear()
        b.clear()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            b.run()
        a.run()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(a.outputs(), want[0]))
        assert all(torch.equal(x, y) for x, y in zip(b.outputs(), want[1]))


def test_route_and_experts_layer_captured(lib):
    """The router's choice and the layer it feeds, replayed with new tokens."""
    T, E, k, D, H = 12, 16, 4, 136, 72
    c = experts_case(lib, T, E, k, D, H, "bf16", "e4m3")
    logits = draw((T, E), "f32", 5).to(DEV)

    def run():
        lib.gemm_experts_route(T, E, logits.data_ptr(), E, lib.INPUT_F32, 0, 0, lib.SCORE_SOFTMAX, 1, 1, 1, k, True, 1.0,
                               c["dids"].data_ptr(), c["dgates"].data_ptr())
        experts_call(lib, c)
    graph = torch.cuda.CUDAGraph()
    run()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        run()
    for seed in (6, 7, 8):
        logits.copy_(draw((T, E), "f32", seed))
        c["my"].view.fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        order = torch.sort(logits.cpu(), dim=1, descending=True, stable=True)
        assert torch.equal(c["dids"].cpu(), order.indices[:, :k].int())
        want, bound = ref.experts_layer(c["x"], c["dids"].cpu(), c["dgates"].cpu(), *c["values"], "silu", 0.0, None, "bf16", "bf16")
        close(c["my"].get(), want, bound, "Y")


def test_orthogonalize_many_matrices(lib):
    """More matrices than one launch takes, of a size that takes several launches a step."""
    M, N, batch = 129, 129, 65600
    few = torch.randn(4, M, N, generator=torch.Generator().manual_seed(8)).bfloat16().to(DEV)
    g = few.repeat(batch // 4, 1, 1)
    o = torch.empty_like(g)
    ws = space(lib.orthogonalize_workspace_size(M, N, batch))
    lib.gemm_orthogonalize(M, N, g.data_ptr(), N, 1, 1, None, 1e-7, 1.0, 0.0, o.data_ptr(), N, 1, ws.data_ptr(), ws.numel() * 4,
                           batch=batch, stride_g=M * N, stride_o=M * N)
    torch.cuda.synchronize()
    for b in range(4):
        want = ref.newton_schulz(few[b].cpu(), 1, None, 1e-7)
        drift = torch.linalg.matrix_norm(ref.newton_schulz(few[b].cpu(), 1, None, 1e-7, rounding=True) - want)
        # as for few matrices; every copy is off by no more
        off = torch.linalg.matrix_norm(o[b::4].double() - want.to(DEV)).max().item()
        assert off <= 2 * drift + (2.0 ** -16 + ref.HALF["bf16"]) * torch.linalg.matrix_norm(want)


@pytest.mark.parametrize("M,N,K", [(1030, 1101, 515), (300, 33030, 520), (40, 300, 1000)])
def test_linear_backward_captured(lib, M, N, K):
    """Copies, tiles left over and slices from a graph, replayed on new inputs: as called, whatever the workspace held."""
    a, b, z = (torch.empty(s, dtype=torch.float16, device=DEV) for s in ((M, K), (N, K), (M, N)))
    d, db = torch.empty_like(z), torch.empty(N, device=DEV)
    ws = space(lib.linear_workspace_size(M, N, K))

    def call(stream=None):
        lib.gemm_linear_backward(M, N, K, 1.0, a.data_ptr(), K, b.data_ptr(), K, lib.COL_MAJOR, 2, z.data_ptr(), N, 2, d.data_ptr(), N, 2,
                                 0.0, db.data_ptr(), ws.data_ptr(), ws.numel() * 4, stream=stream)

    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    for t in (a, b, z):
        t.zero_()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        call(torch.cuda.current_stream().cuda_stream)
    for seed in range(3):
        g = torch.Generator(device=DEV).manual_seed(seed)
        for t in (a, b, z):
            t.normal_(generator=g)
        ws.fill_(float("nan") if ws.is_floating_point() else -1)
        graph.replay()
        torch.cuda.synchronize()
        got = d.clone(), db.clone()
        ws.fill_(0)
        d.fill_(9), db.fill_(9)
        call(torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert torch.equal(got[0], d) and torch.equal(got[1], db)
        assert got[0].isfinite().all() and got[1].isfinite().all()


# ---------------------------------------------------------------- infinities and NaN through the activations
ACT = {"none": 0, "relu": 1, "gelu": 2, "silu": 3}
# few rows; tiles; tiles through registers; slices of tiles; no product
KERNEL_SIZES = [(5, 40, 64), (130, 136, 128), (30, 75, 99), (40, 300, 1000), (9, 44, 0)]
BIG = {"bf16": 3e38, "f16": 6e4}


def linear_of_bias(lib, M, N, K, kind, act, bias):
    """gemm_linear's C in fp32 and Z of small products and this bias."""
    a, b = draw((M, K), kind, 1, 0.1), draw((N, K), kind, 2, 0.1)
    da, db, dbias = a.to(DEV), b.to(DEV), bias.to(ref.TORCH[kind]).to(DEV)
    c, z = torch.zeros(M, N, device=DEV), torch.zeros(M, N, dtype=ref.TORCH[kind], device=DEV)
    ws = space(lib.linear_workspace_size(M, N, K))
    lib.gemm_linear(M, N, K, 1.0, da.data_ptr(), K, db.data_ptr(), K, 1, INPUT[kind], dbias.data_ptr(), ACT[act], 0.0, 0, 0,
                    c.data_ptr(), N, 0, z.data_ptr(), N, ws.data_ptr(), ws.numel() * 4)
    torch.cuda.synchronize()
    return c.cpu().double(), z.cpu().double(), a.double() @ b.double().t() + bias.to(ref.TORCH[kind]).double()


def slope_of(lib, M, N, K, kind, act, z, incoming):
    """gemm_linear_backward's D in fp32 and its column sums: row i of the gradient is incoming[i] in every column."""
    k = max(K, 1)
    a, b = torch.zeros(M, k, dtype=ref.TORCH[kind]), torch.zeros(N, k, dtype=ref.TORCH[kind])
    a[:, 0], b[:, 0] = incoming.to(a.dtype), 1
    da, db, dz = a.to(DEV), b.to(DEV), z.to(ref.TORCH[kind]).to(DEV)
    d, sums = torch.zeros(M, N, device=DEV), torch.zeros(N, device=DEV)
    ws = space(lib.linear_workspace_size(M, N, k))
    lib.gemm_linear_backward(M, N, k, 1.0, da.data_ptr(), k, db.data_ptr(), k, 1, INPUT[kind], dz.data_ptr(), N, ACT[act],
                             d.data_ptr(), N, 0, 0.0, sums.data_ptr(), ws.data_ptr(), ws.numel() * 4)
    torch.cuda.synchronize()
    return d.cpu().double(), sums.cpu().double()


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", KERNEL_SIZES)
def test_relu_keeps_nan(lib, M, N, K, kind):
    """A NaN passes ReLU, and its slope there is NaN: nothing turns one into a 0."""
    bias = torch.zeros(N)
    bias[3], bias[N - 1] = float("nan"), float("nan")
    c, z, pre = linear_of_bias(lib, M, N, K, kind, "relu", bias)
    assert torch.equal(z.isnan(), pre.isnan()) and torch.equal(c.isnan(), pre.isnan())
    d, sums = slope_of(lib, M, N, K, kind, "relu", pre, torch.ones(M))
    assert torch.equal(d.isnan(), pre.isnan()) and torch.equal(sums.isnan(), pre.isnan().any(0))


@pytest.mark.parametrize("act", ["relu", "gelu", "silu"])
def test_experts_layer_keeps_nan(lib, act):
    """A NaN among an expert's activated weights reaches every token that chose it, and no other."""
    ids = torch.tensor([[0, 1], [2, 3], [1, 2], [3, 0]], dtype=torch.int32)
    c = experts_case(lib, 4, 4, 2, 72, 40, act=act, ids=ids)
    c["stored"][0][0][1, 7, 5] = float("nan")
    experts_call(lib, c)
    torch.cuda.synchronize()
    want, bound = ref.experts_layer(c["x"], ids, c["gates"], *c["values"], act, 0.0, None, "bf16", "bf16")
    got = c["my"].get()
    assert got[[0, 2]].isnan().all()
    close(got[[1, 3]], want[[1, 3]], bound[[1, 3]], "Y")


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", KERNEL_SIZES)
def test_relu_slope_is_a_choice(lib, M, N, K, kind):
    """Where ReLU was off its gradient is 0, whatever comes in: infinities and NaN there do not reach D or its sums."""
    z = draw((M, N), kind, 3).double()
    z[:, 1], z[:, 2] = 0.0, -0.0
    incoming = torch.ones(M)
    incoming[1], incoming[2], incoming[4] = float("inf"), float("nan"), -float("inf")
    z[[1, 2, 4], :6] = -z[[1, 2, 4], :6].abs()
    d, sums = slope_of(lib, M, N, K, kind, "relu", z, incoming)
    want = torch.where(z > 0, incoming.double()[:, None], 0.0)
    assert torch.equal(d.nan_to_num(nan=9.0), want.nan_to_num(nan=9.0))
    # whole numbers where every term is finite
    assert torch.equal(sums[:6], want[:, :6].sum(0))
    dz, da = z.to(ref.TORCH[kind]).to(DEV), incoming.to(ref.TORCH[kind])[:, None].repeat(1, N).to(DEV)
    out, total = torch.zeros(M, N, device=DEV), torch.zeros(N, device=DEV)
    ws = space(lib.activation_backward_workspace_size(M, N))
    lib.gemm_activation_backward(M, N, da.data_ptr(), N, INPUT[kind], dz.data_ptr(), N, INPUT[kind], lib.ACT_RELU, out.data_ptr(), N,
                                 0, 0.0, total.data_ptr(), ws.data_ptr(), ws.numel() * 4)
    torch.cuda.synchronize()
    assert torch.equal(out.cpu().double().nan_to_num(nan=9.0), want.nan_to_num(nan=9.0))
    assert torch.equal(total[:6].cpu().double(), want[:, :6].sum(0))


@pytest.mark.parametrize("act", ["gelu", "silu"])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", KERNEL_SIZES)
def test_activations_at_infinity(lib, M, N, K, kind, act):
    """GELU and SiLU take their limits at infinities (0 and +inf; slopes 0 and 1), where fp16's Z of a large value is one; NaN
    stays NaN; the tails in between are as near as anywhere."""
    special = [float("nan"), float("inf"), -float("inf"), BIG[kind], -BIG[kind], 30.0, -30.0, -12.0, -9.0, 100.0, -100.0]
    bias = torch.zeros(N)
    bias[:len(special)] = torch.tensor(special)
    c, z, pre = linear_of_bias(lib, M, N, K, kind, act, bias)
    want = torch.where(pre == -float("inf"), 0.0, ref.act(pre, act))
    assert torch.equal(c.isnan(), want.isnan()) and torch.equal(c.isinf(), want.isinf())
    assert c[:, 0].isnan().all() and (c[:, 1] == float("inf")).all() and (c[:, 2] == 0).all()
    fine = pre.isfinite()  # the others are compared above
    # |product| < 30: fp32's sums are off by 2^-23 of K + 8 such terms at most, and of z itself; no slope passes 1.13
    error = 1.13 * ((K + 8) * 30 * 2.0 ** -23 * 0.01 + 2.0 ** -23 * pre.abs()) + ref.act_error(pre, act)
    close(c[fine], want[fine], (error * 1.01 + 2.0 ** -24 * want.abs() + 2.0 ** -126)[fine], "C")
    d, sums = slope_of(lib, M, N, K, kind, act, z, torch.ones(M))
    s = torch.where(z == float("inf"), 1.0, torch.where(z == -float("inf"), 0.0, ref.slope(z, act)))
    assert torch.equal(d.isnan(), s.isnan()) and torch.equal(sums.isnan(), s.isnan().any(0)) and not d.isinf().any()
    fine = z.isfinite()
    close(d[fine], s[fine], (ref.slope_error(z, act) + 2.0 ** -22 * s.abs() + 2.0 ** -126)[fine], "D")
    assert (d[:, 1] == 1).all() and (d[:, 2] == 0).all()


@pytest.mark.parametrize("alpha", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("M,N", [(3, 17), (130, 264)])
def test_empty_product_whatever_alpha(lib, M, N, alpha):
    """K = 0: there is nothing for alpha to scale."""
    run_linear(lib, M, N, 0, alpha=1.0, beta=1.0, keep=True)
    bi, z = draw((N,), "bf16", 4), draw((M, N), "bf16", 5)
    b, dz = bi.to(DEV), z.to(DEV)
    c, kept = torch.zeros(M, N, device=DEV), torch.zeros(M, N, dtype=torch.bfloat16, device=DEV)
    lib.gemm_linear(M, N, 0, alpha, 0, 0, 0, 0, 1, 1, b.data_ptr(), 0, 0.0, 0, 0, c.data_ptr(), N, 0, kept.data_ptr(), N)
    d, sums = torch.ones(M, N, device=DEV), torch.arange(N, dtype=torch.float32, device=DEV)
    ws = space(lib.linear_workspace_size(M, N, 0))
    lib.gemm_linear_backward(M, N, 0, alpha, 0, 0, 0, 0, 1, 1, dz.data_ptr(), N, 2, d.data_ptr(), N, 0, 0.5, sums.data_ptr(),
                             ws.data_ptr(), ws.numel() * 4)
    torch.cuda.synchronize()
    assert torch.equal(c, b.float().expand(M, N)) and torch.equal(kept, b.expand(M, N))
    assert not d.any() and torch.equal(sums.cpu(), torch.arange(N, dtype=torch.float32) / 2)


@pytest.mark.parametrize("ratio", [1e-2, 1e-4, 1e-6, 1e-8, 1e-12, 1e-20])
@pytest.mark.parametrize("M,N,kernel", [(60, 90, "orthogonalize_small"), (150, 200, "orthogonalize_mfma_128_few"),
                                        (260, 140, "orthogonalize_mfma_128_few")])
def test_orthogonalize_norms_below_eps(lib, M, N, kernel, ratio):
    """A norm far below eps: X starts as small and grows by a factor of 3.45 a step at most, and keeps its digits."""
    assert lib.orthogonalize_kernel_name(M, N, 1) == kernel
    steps = 5
    x = matrix(M, N, 3, "plain").float()
    eps = torch.tensor(torch.linalg.matrix_norm(x.double()).item() / ratio, dtype=torch.float32).item()
    d, o = x.to(DEV), torch.zeros(M, N, device=DEV)
    ws = space(lib.orthogonalize_workspace_size(M, N, 1))
    lib.gemm_orthogonalize(M, N, d.data_ptr(), N, 0, steps, None, eps, 1.0, 0.0, o.data_ptr(), N, 0, ws.data_ptr(), ws.numel() * 4)
    torch.cuda.synchronize()
    want = ref.newton_schulz(x, steps, None, eps)
    size = torch.linalg.matrix_norm(want).item()
    # B X with three roundings of 2^-11 each, |B| < 4.8 |X|^2 and |X| < ratio * 3.45^4 before the last step; the four before
    # add less than that again (|X|^2 is 12 times smaller each time).  X itself: each step rounds it to 22 bits, or in steps of
    # 2^-24 where its norm is 2^9 or more, 190 root mean squares: below 2^-20 a step.  fp32's own: below 2^-18 over all
    largest = min(1.0, ratio * 3.45 ** (steps - 1))
    bound = size * (2 * 4.8 * largest ** 2 * 3 * 2.0 ** -11 + steps * 2.0 ** -20 + 2.0 ** -18)
    assert torch.linalg.matrix_norm(o.cpu().double() - want).item() <= bound


def test_orthogonalize_norms_of_a_batch(lib):
    """Each matrix of a batch has a scale of its own; coefficients as large as the call promises to hold."""
    M, N, steps = 150, 200, 3
    coefficients = [(15.0, 15.0, -15.0), (2.0, -1.5, 0.5), (2.0, -1.5, 0.5)]
    x = torch.stack([matrix(M, N, 5 + b, "plain") for b in range(4)])
    x = x / torch.linalg.matrix_norm(x)[:, None, None]
    x = (x * torch.tensor([1e-9, 0.01, 0.06, 0.0], dtype=torch.float64)[:, None, None]).float()
    d, o = x.to(DEV), torch.zeros(4, M, N, device=DEV)
    ws = space(lib.orthogonalize_workspace_size(M, N, 4))
    assert lib.orthogonalize_kernel_name(M, N, 4) != "orthogonalize_small"
    lib.gemm_orthogonalize(M, N, d.data_ptr(), N, 0, steps, coefficients, 1.0, 1.0, 0.0, o.data_ptr(), N, 0, ws.data_ptr(),
                           ws.numel() * 4, batch=4, stride_g=M * N, stride_o=M * N)
    torch.cuda.synchronize()
    for b, norm in enumerate((1e-9, 0.01, 0.06)):
        want = ref.newton_schulz(x[b], steps, coefficients, 1.0)
        size = torch.linalg.matrix_norm(want).item()
        # |B| < 16 |X|^2 in the first step, then 1.6 |X|^2 of an X up to 15.1 and 31 times larger; roundings as above
        bound = size * (2 * 3 * 2.0 ** -11 * (16 * norm ** 2 + 1.6 * (15.1 * norm) ** 2 + 1.6 * min(1.0, 31 * norm) ** 2) +
                        steps * 2.0 ** -20 + 2.0 ** -18)
        assert torch.linalg.matrix_norm(o[b].cpu().double() - want).item() <= bound
    assert not o[3].any()


@pytest.mark.parametrize("form", ["same", "e4m3"])
@pytest.mark.parametrize("gate,weight", [(2.0 ** -14, 64.0), (2.0 ** -20, 1024.0), (2.0 ** 18, 1.0)])
def test_experts_layer_range_of_products(lib, form, gate, weight):
    """fp16's w h from 2^-30 to 2^19.4, far below its smallest normal value and beyond its largest, for an fp32 Y."""
    T, E, k, D, H = 9, 4, 2, 136, 200
    c = experts_case(lib, T, E, k, D, H, "f16", form, act="relu", out="f32")
    c["gates"] *= gate
    c["dgates"].copy_(c["gates"])
    down = c["stored"][1]
    (down[0] if form == "same" else down[1]).mul_(weight)
    c["values"][1] = [v * weight for v in c["values"][1]]
    experts_call(lib, c)
    torch.cuda.synchronize()
    want, bound = ref.experts_layer(c["x"], c["ids"], c["gates"], *c["values"], "relu", 0.0, None, "f32", "f16")
    # the reference allows steps of 2^-24 in w h; they are 2^-31 (2^4 times fp16's 2^-24 times 2^-11)
    size = torch.stack([sum(c["values"][1][e].abs().sum(1) for e in row.tolist()) for row in c["ids"]])
    bound = bound - (2.0 ** -24 - 2.0 ** -31) * size
    assert (bound > 0).all()
    close(c["my"].get(), want, bound, "Y")


# ---------------------------------------------------------------- more stages than a ring holds
@pytest.mark.parametrize("M,N,K,kind", [(1, 40, 10000, "bf16"), (4, 33, 8200, "f16"), (7, 50, 10000, "f16"), (8, 16, 12296, "bf16"),
                                        (9, 70, 10000, "bf16"), (16, 100, 8200, "f16"), (16, 48, 16384, "bf16")])
@pytest.mark.parametrize("backward", [False, True])
def test_linear_few_rows_long_k(lib, M, N, K, kind, backward):
    """Each wave of few_kernel has 8 to 16 runs of K, its ring 2 to 4; the last runs are partial."""
    if backward:
        run_backward(lib, M, N, K, kind, expect="linear_few_16", beta=1.0)
    else:
        run_linear(lib, M, N, K, kind, beta=1.0, keep=True, expect="linear_few_16")


@pytest.mark.parametrize("kind,order", [("bf16", "nk"), ("f16", "kn"), ("bf16", "kn")])
@pytest.mark.parametrize("backward", [False, True])
def test_linear_large_tiles_long_k(lib, kind, order, backward):
    """256 x 256 tiles whose two stages are refilled; the last stage is partial."""
    M, N, K = 3600, 3656, 584
    if backward:
        run_backward(lib, M, N, K, kind, order, expect="linear_mfma_256")
    else:
        run_linear(lib, M, N, K, kind, order, beta=1.0, keep=True, out="f32", expect="linear_mfma_256")


@pytest.mark.parametrize("form,kind", [("same", "bf16"), ("same", "f16"), ("e4m3", "bf16"), ("e5m2", "f16"), ("e4m3", "f16")])
@pytest.mark.parametrize("T,E,k,H", [(1, 4, 2, 1000), (3, 8, 2, 1000), (12, 8, 2, 1000), (32, 6, 2, 1000), (20, 2, 2, 2056)])
def test_experts_layer_long_rows(lib, T, E, k, H, form, kind):
    """D = 4104: each wave has 4 to 9 runs of a row, more blocks than one, and groups of one expert and the next in a workgroup;
    H is 8 to 33 runs of each of several experts.  T by 8 and by 16 tokens at a time, and by 4 and 8."""
    experts_check(lib, T, E, k, 4104, H, kind, form, beta=1.0)


# ---------------------------------------------------------------- special values of matrices that take several launches
LARGE = [(150, 200), (260, 140)]  # one as it is, one turned


def several_launches(lib, M, N, batch=1):
    assert lib.orthogonalize_kernel_name(M, N, batch).startswith("orthogonalize_mfma")


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e-12, 1.0, 1e15, 1e30, 1e36])
@pytest.mark.parametrize("M,N", LARGE)
def test_orthogonalize_scales_of_large(lib, M, N, scale, kind):
    """As test_orthogonalize_scales; the smallest are subnormal."""
    several_launches(lib, M, N)
    run_ortho(lib, M, N, kind, scale=scale, eps=0.0)


@pytest.mark.parametrize("M,N", LARGE)
def test_orthogonalize_unusual_values_of_large(lib, M, N):
    """As test_orthogonalize_unusual_values."""
    several_launches(lib, M, N, 5)
    x = torch.stack([matrix(M, N, i, "plain") for i in range(5)]).float()
    x[0], x[1, 5, 6], x[2, 3, 3], x[4, M - 1, N - 1] = 0, float("inf"), float("nan"), -float("inf")
    d, o = x.to(DEV), torch.ones(5, M, N, device=DEV)
    ws = space(lib.orthogonalize_workspace_size(M, N, 5))
    for eps in (0.0, 1e-7):
        o.fill_(1)
        lib.gemm_orthogonalize(M, N, d.data_ptr(), N, 0, 5, None, eps, 1.0, 0.5, o.data_ptr(), N, 0, ws.data_ptr(), ws.numel() * 4,
                               batch=5, stride_g=M * N, stride_o=M * N)
        torch.cuda.synchronize()
        assert (o[0] == 0.5).all() and o[1].isnan().all() and o[2].isnan().all() and o[4].isnan().all()
        want = ref.newton_schulz(x[3], 5)
        drift = torch.linalg.matrix_norm(ref.newton_schulz(x[3], 5, rounding=True) - want)
        off = torch.linalg.matrix_norm(o[3].cpu().double() - 0.5 - want)
        # as run_ortho's bound; the halves of O round to 2^-24
        assert off <= 2 * drift + 2.0 ** -16 * torch.linalg.matrix_norm(want) + 2.0 ** -24 * (M * N) ** 0.5


@pytest.mark.parametrize("M,N", LARGE)
def test_orthogonalize_steps_of_large(lib, M, N):
    """As test_orthogonalize_coefficients, and every number of steps (X's two buffers change places in each)."""
    several_launches(lib, M, N)
    cubic = [(4.0848, -6.8946, 2.9270), (3.9505, -6.3029, 2.6377), (3.7418, -5.5913, 2.3037), (2.8769, -3.1427, 1.2046),
             (2.8366, -3.0525, 1.2012), (1.5, -0.5, 0.0), (1.5, -0.5, 0.0), (1.5, -0.5, 0.0)]
    x = run_ortho(lib, M, N, steps=8, coefficients=cubic)[0]
    assert (torch.linalg.svdvals(x) - 1).abs().max() < 0.02
    for steps in (1, 2, 3, 4, 32):
        run_ortho(lib, M, N, steps=steps, coefficients=[(1.5, -0.5, 0.0)] * steps, beta=0.5)


# ---------------------------------------------------------------- tokens among others
@pytest.mark.parametrize("form,kind", [("same", "f16"), ("e4m3", "bf16")])
@pytest.mark.parametrize("T,E", [(6, 4), (40, 3)])
def test_experts_layer_unusual_tokens(lib, T, E, form, kind):
    """A token with an infinity or a NaN leaves those it shares experts, and matrix instructions, with as they were."""
    c = experts_case(lib, T, E, 2, 200, 136, kind, form)
    c["x"][2, 7], c["x"][5, 199], c["x"][T - 1, 0] = float("nan"), float("inf"), float("nan")
    c["mx"].view.copy_(c["x"])
    c["dgates"][0, 0] = float("inf")
    experts_call(lib, c)
    torch.cuda.synchronize()
    odd = sorted({0, 2, 5, T - 1})
    fine = [t for t in range(T) if t not in odd]
    want, bound = ref.experts_layer(c["x"], c["ids"], c["gates"], *c["values"], "silu", 0.0, None, kind, kind)
    got = c["my"].get()
    assert not got[odd].isfinite().any()
    close(got[fine], want[fine], bound[fine], "Y")
