"""CPU pins of the MXFP4 oracle (E2M1 codes, block exponents, packing, block norms) and the
host-side refusals of the MXFP4 and block-norm entry points."""

import ctypes
import itertools

import numpy as np
import pytest

import oracle as O

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def test_e2m1_values():
    assert O.e2m1_decode(np.arange(16)).tolist() == E2M1 + [-v for v in E2M1]


def test_e2m1_ties_go_to_the_even_code():
    ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    assert O.e2m1_encode(np.float32(ties)).tolist() == [0, 2, 2, 4, 4, 6, 6]
    assert O.e2m1_encode(-np.float32(ties)).tolist() == [8, 10, 10, 12, 12, 14, 14]
    assert O.e2m1_encode(np.float32([-0.0, 0.0, -0.1, -1e-45])).tolist() == [8, 0, 8, 8]


def test_e2m1_nearest_by_search():
    x = np.random.default_rng(0).uniform(-6, 6, 20000).astype(np.float32)
    v = np.array(E2M1)
    want = np.abs(np.abs(x)[:, None].astype(np.float64) - v[None, :]).argmin(axis=1)
    assert np.array_equal(O.e2m1_encode(x) & 7, want)


def test_exponent_is_the_smallest_that_does_not_clip():
    a = np.float32([6.0, 6.0000005, 3.0, 3.1, 12.0, 1e-30, 2.0 ** -149, 3.4e38])
    X = O.mxfp4_exponent(a).astype(np.int64)
    a64 = a.astype(np.float64)
    assert np.all(a64 <= 6.0 * 2.0 ** X)
    assert np.all((a64 > 6.0 * 2.0 ** (X - 1)) | (X == -127))
    assert O.mxfp4_exponent(0.0) == -127
    assert X.tolist()[:5] == [0, 1, -1, 0, 1]


def test_quantize_rows_and_packing():
    A = np.zeros((2, 64), np.float32)
    A[0, :4] = [6.0, -3.0, 0.5, -0.2]
    A[1, 33] = np.nan
    codes, X = O.mxfp4_quantize_rows(A)
    assert codes[0, :4].tolist() == [7, 13, 1, 8]
    assert X.tolist() == [[0, -127], [-127, 128]]
    assert O.mxfp4_pack(codes)[0, :2].tolist() == [7 | (13 << 4), 1 | (8 << 4)]
    v = O.mx_values(codes, X, "mxfp4")
    assert v[0, :4].tolist() == [6.0, -3.0, 0.5, -0.0]
    assert np.isnan(v[1, 32:]).all() and not np.isnan(v[1, :32]).any()


def test_error_of_a_value_is_at_most_half_a_step_of_its_binade():
    # |v| 2^-X in (2, 6]: steps of at most 2, so off by at most 1 in units of 2^X
    A = np.random.default_rng(1).standard_normal((16, 320)).astype(np.float32)
    codes, X = O.mxfp4_quantize_rows(A)
    v = O.mx_values(codes, X, "mxfp4")
    step = 2.0 ** np.repeat(X.astype(np.float64), 32, axis=1)
    assert np.all(np.abs(v - A) <= step)


def test_block_norm_against_plain_float64():
    rng = np.random.default_rng(3)
    M, K = 5, 96
    Y, H = (O.f32_to_bf16_bits(rng.standard_normal((M, K)).astype(np.float32)) for _ in range(2))
    g, pg, gate = (rng.uniform(0.5, 1.5, K).astype(np.float32) for _ in range(3))
    b, pb = (rng.standard_normal(K).astype(np.float32) for _ in range(2))
    for kind in ("rms", "layer"):
        hb, z = O.block_norm(Y, H, g, pg, gate, 0.5, b, pb, 1e-6, kind)

        def norm(x, g, b):
            if kind == "layer":
                x = x - x.mean(axis=1, keepdims=True)
            return x / np.sqrt((x * x).mean(axis=1, keepdims=True) + 1e-6) * g + b

        y = norm(O.bf16_bits_to_f32(Y).astype(np.float64), pg, pb) * gate
        h = 0.5 * O.bf16_bits_to_f32(H).astype(np.float64) + y
        got = O.bf16_bits_to_f32(hb).astype(np.float64)
        # bf16 rounding, and a few fp32 roundings of terms below 8
        assert np.all(np.abs(got - h) <= 2.0 ** -8 * np.abs(h) + 8 * 2.0 ** -21)
        # against float64 from the rounded h': the mean (layer) and r are rounded to fp32
        # once, then at most four fp32 operations on terms below 8
        assert np.all(np.abs(z - norm(got, g, b)) <= 8 * 8 * 2.0 ** -24)


# ----------------------------------------------------------------------------
# Host-side refusals (every call below fails before any HIP call)
# ----------------------------------------------------------------------------

@pytest.fixture(scope="module")
def L():
    from w8a8_gemm_rl_amd import binding
    return binding.lib()


F = ctypes.c_void_p(1 << 20)
MX8, MX4 = 2, 3


def _call(f, spec, **kw):
    assert set(kw) <= set(k for k, _ in spec), kw
    return f(*[kw.get(k, v) for k, v in spec])


def test_quantize_refusals(L):
    spec = [("A", F), ("R", 4), ("K", 64), ("lda", 64), ("bf16", 1), ("codes", F), ("scales", F), ("st", None)]
    q = lambda **kw: _call(L.qr_mxfp4_quantize, spec, **kw)  # noqa: E731
    assert q(R=-1) == -1 and q(K=-32) == -1 and q(R=1 << 31) == -1
    assert q(bf16=2) == -1
    assert q(K=48) == -2
    assert q(lda=32) == -1
    assert q(lda=68) == -2 and q(lda=66, bf16=0) == -2
    for k in ("A", "codes", "scales"):
        assert q(**{k: None}) == -1
    assert q(A=ctypes.c_void_p(8)) == -2 and q(codes=ctypes.c_void_p(8)) == -2
    assert q(scales=ctypes.c_void_p(2)) == -2
    assert b"qr_mxfp4_quantize" in L.qr_last_error()


def test_dequantize_refusals(L):
    spec = [("codes", F), ("scales", F), ("R", 4), ("K", 64), ("fmt", MX4), ("out", F), ("ldo", 64), ("bf16", 1),
            ("st", None)]
    d = lambda **kw: _call(L.qr_mx_dequantize, spec, **kw)  # noqa: E731
    for fmt in (-1, 0, 1, 4):
        assert d(fmt=fmt) == -1
    assert d(R=-1) == -1 and d(bf16=3) == -1 and d(ldo=63) == -1 and d(out=None) == -1
    assert d(K=16, ldo=16) == -2 and d(ldo=66, bf16=0) == -2 and d(ldo=68) == -2
    assert d(out=ctypes.c_void_p(4)) == -2


def test_product_refusals(L):
    spec = [("Xq", F), ("sx", F), ("xfmt", MX4), ("Wq", F), ("sw", F), ("M", 4), ("N", 64), ("K", 256), ("out", 0),
            ("Y", F), ("ldy", 64), ("ws", None), ("wsb", 0), ("st", None)]
    g = lambda **kw: _call(L.qr_mxfp4_gemm, spec, **kw)  # noqa: E731
    for x in (0, 1, 4, 7):
        assert g(xfmt=x) == -1
    assert g(M=-1) == -1 and g(N=1 << 31) == -1 and g(out=2) == -1 and g(ldy=63) == -1
    for k in ("Xq", "sx", "Wq", "sw", "Y"):
        assert g(**{k: None}) == -1
        assert g(**{k: ctypes.c_void_p(8)}) == -2
    assert g(K=64) == -2 and g(K=160) == -2
    assert g(N=1 << 20, K=4096, ldy=1 << 20) == -2  # 2^31 bytes of codes
    assert g(M=1 << 19, K=4096, xfmt=MX8) == -2
    spec = [("X", F), ("ldx", 256), ("xfmt", MX4), ("Wq", F), ("sw", F), ("M", 4), ("N", 64), ("K", 256), ("Y", F),
            ("ldy", 64), ("ws", F), ("wsb", 1 << 20), ("st", None)]
    li = lambda **kw: _call(L.qr_mxfp4_linear, spec, **kw)  # noqa: E731
    assert li(xfmt=1) == -1 and li(ldx=255) == -1 and li(X=None) == -1 and li(Y=None) == -1
    assert li(ldx=260) == -2 and li(X=ctypes.c_void_p(8)) == -2 and li(K=128 + 64) == -2
    big = dict(M=100, K=1024, ldx=1024)
    assert li(ws=None, **big) == -3 and li(wsb=16, **big) == -3
    assert li(ws=ctypes.c_void_p((1 << 20) + 64), **big) == -3
    assert li(M=1 << 20, N=1 << 18, ldy=1 << 18, K=128) == -2  # M N = 2^38


def test_workspace_sizes(L):
    ws = L.qr_workspace_size
    none = ctypes.c_size_t(-1).value
    for fn, x in itertools.product((b"qr_mxfp4_gemm", b"qr_mxfp4_linear"), (MX8, MX4)):
        assert ws(fn, 0, 64, 256, x) == 0 and ws(fn, 4, 0, 256, x) == 0
        assert ws(fn, 4, 64, 200, x) == none and ws(fn, -1, 64, 256, x) == none
        assert ws(fn, 4, 64, 256, 0) == none
    # the linear holds codes and scales besides what its product needs
    for x, per in ((MX8, 1.0), (MX4, 0.5)):
        need = ws(b"qr_mxfp4_linear", 33, 512, 1024, x) - ws(b"qr_mxfp4_gemm", 33, 512, 1024, x)
        assert need >= 33 * 1024 * per + 33 * 32
        # a few tokens are quantized inside the kernel
        assert ws(b"qr_mxfp4_linear", 1, 512, 18944, x) == 0 and ws(b"qr_mxfp4_linear", 16, 512, 1024, x) == 0
        assert ws(b"qr_mxfp4_linear", 1, 512, 41088, x) > 0 and ws(b"qr_mxfp4_linear", 17, 512, 128, x) > 0


def test_block_norm_refusals(L):
    G = lambda i: ctypes.c_void_p((i + 1) << 20)  # noqa: E731  (rows apart from each other)
    spec = [("Y", G(0)), ("ldy", 64), ("H", G(1)), ("ldh", 64), ("M", 4), ("K", 64), ("norm", 0), ("pg", G(2)),
            ("pb", None), ("gate", None), ("ldg", 0), ("res", 1.0), ("gamma", G(3)), ("beta", None), ("eps", 1e-6),
            ("fmt", MX4), ("Hout", G(4)), ("ldo", 64), ("codes", G(5)), ("scales", G(6)), ("st", None)]
    b = lambda **kw: _call(L.qr_block_norm_quant, spec, **kw)  # noqa: E731
    assert b(M=-1) == -1 and b(norm=2) == -1 and b(fmt=5) == -1 and b(fmt=-1) == -1
    for v in (float("nan"), float("inf"), -1.0):
        assert b(eps=v) == -1
    assert b(res=float("inf")) == -1 and b(res=float("nan")) == -1
    assert b(pg=None, pb=G(7)) == -1
    assert b(K=48) == -2 and b(K=24, fmt=0) == -2 and b(K=32800, ldy=32800, ldh=32800, ldo=32800) == -2
    for k in ("ldy", "ldh", "ldo"):
        assert b(**{k: 32}) == -1
        assert b(**{k: 68}) == -2
    assert b(gate=G(8), ldg=32) == -1 and b(gate=G(8), ldg=68) == -2
    for k in ("Y", "H", "gamma", "Hout", "codes", "scales"):
        assert b(**{k: None}) == -1
    for k in ("Y", "H", "pg", "gamma", "Hout", "codes"):
        assert b(**{k: ctypes.c_void_p(8)}) == -2
    # Hout over part of H, over Y at another stride, over a shifted row
    H = G(1).value
    assert b(Hout=ctypes.c_void_p(H + 32)) == -1
    assert b(Hout=ctypes.c_void_p(H), ldo=128) == -1
    assert b(Hout=ctypes.c_void_p(H + 128)) == -1
    assert b(gate=G(8), ldg=64, Hout=ctypes.c_void_p(G(8).value + 16)) == -1
    assert b"overlaps" in L.qr_last_error()


def test_silu_refusals(L):
    spec = [("G", F), ("U", F), ("M", 4), ("N", 64), ("ldg", 64), ("ldu", 64), ("fmt", MX4), ("codes", F),
            ("scales", F), ("st", None)]
    s = lambda **kw: _call(L.qr_silu_mul_mx, spec, **kw)  # noqa: E731
    assert s(fmt=1) == -1 and s(fmt=4) == -1 and s(M=-1) == -1 and s(ldg=32) == -1 and s(ldu=32) == -1
    assert s(N=48) == -2 and s(ldg=68) == -2 and s(codes=ctypes.c_void_p(8)) == -2
    for k in ("G", "U", "codes", "scales"):
        assert s(**{k: None}) == -1


def test_binding_refuses_host_tensors_and_bad_types():
    import torch
    from w8a8_gemm_rl_amd import binding as B

    w = torch.zeros((4, 64), dtype=torch.uint8)
    s = torch.zeros((1, 4, 4), dtype=torch.uint8)
    x = torch.zeros((2, 128), dtype=torch.bfloat16)
    for f in (lambda: B.mxfp4_quantize(x), lambda: B.mx_dequantize(w, s), lambda: B.mxfp4_linear(x, w, s),
              lambda: B.mxfp4_gemm(w, s, w, s), lambda: B.silu_mul_mx(x, x, "mxfp4"),
              lambda: B.block_norm_quant(x, x, torch.ones(128), "mxfp4")):
        with pytest.raises(ValueError, match="HIP device"):
            f()


def test_binding_passes_the_row_stride_of_an_output_as_it_is():
    """A stride below N (an expanded row) reaches the library, which refuses it."""
    import torch
    from w8a8_gemm_rl_amd import binding as B

    like = torch.zeros((1,), dtype=torch.bfloat16)
    y = torch.zeros((1, 16), dtype=torch.bfloat16)
    assert B._mx4_out(y.expand(4, 16), like, 4, 16, torch.bfloat16)[1] == 0
    assert B._mx4_out(y, like, 1, 16, torch.bfloat16)[1] == 16
    assert B._mx4_out(torch.zeros((4, 20), dtype=torch.bfloat16)[:, :16], like, 4, 16, torch.bfloat16)[1] == 20
    assert B._mx4_out(torch.zeros((3, 0), dtype=torch.bfloat16), like, 3, 0, torch.bfloat16)[1] >= 0


def test_gate_row_strides():
    """A gate per channel is fp32 [K], stride 0 in the library; rows of a bf16 gate that are one row
    expanded, whose stride is 0 as well, must not reach it as that."""
    import torch
    from w8a8_gemm_rl_amd import binding as B

    shape = torch.Size((4, 64))
    row = torch.zeros(64, dtype=torch.bfloat16)
    assert B._gate_ld(torch.zeros(64), shape) == 0
    assert B._gate_ld(torch.zeros(shape, dtype=torch.bfloat16), shape) == 64
    assert B._gate_ld(torch.zeros((4, 80), dtype=torch.bfloat16)[:, :64], shape) == 80
    assert B._gate_ld(row.expand(1, 64), torch.Size((1, 64))) == 64
    for gate in (row.expand(4, 64), row.view(1, 64).expand(4, 64), torch.zeros(256, dtype=torch.bfloat16).as_strided((4, 64), (32, 1))):
        with pytest.raises(B.QRError, match="row stride"):
            B._gate_ld(gate, shape)
    for gate in (row, torch.zeros(shape), torch.zeros(128)[::2], torch.zeros(1).expand(64), torch.zeros((64, 4), dtype=torch.bfloat16).t()):
        with pytest.raises(ValueError):
            B._gate_ld(gate, shape)


def test_plan_refusals(L):
    out = [ctypes.byref(ctypes.c_int()) for _ in range(4)]
    f = L.qr_mxfp4_plan
    assert f(16, 256, 256, MX4, *out) == 0
    assert f(16, 256, 256, 1, *out) == -1 and f(-1, 256, 256, MX4, *out) == -1
    assert f(16, 256, 192, MX4, *out) == -2 and f(1 << 20, 1 << 18, 128, MX8, *out) == -2
    for i in range(4):
        assert f(16, 256, 256, MX4, *[None if j == i else o for j, o in enumerate(out)]) == -1
    assert b"qr_mxfp4_plan" in L.qr_last_error()


@pytest.mark.parametrize("x", ["fp4", "fp8"])
def test_gpu_tests_run_every_plan(x):
    """(tile, whether K is split, whether blocks take several tiles): each that a sweep of shapes
    meets is that of a shape of the GPU tests."""
    import test_gpu_mxfp4 as T
    from w8a8_gemm_rl_amd import binding as B

    def plan(M, N, K):
        n, m, splits, ahead = B.mxfp4_plan(M, N, K, x)
        return n, m, splits > 1, ahead

    run = {plan(*s) for s in T.SHAPES + T.CONFIGS + T.PLANS + [s[:3] for s in T.SEVERAL]}
    rng = np.random.default_rng(7)
    met = set()
    for a, b, c in rng.random((40000, 3)):
        M, N, K = int(2 ** (13.2 * a)), int(2 ** (3 + 13.2 * b)), 128 * int(2 ** (7.6 * c))
        if N * K < 1 << 31:
            met.add(plan(M, N, K))
    assert len(met) >= 18 and met <= run, sorted(met - run)
    # one kernel without token tiles, and each tile with and without a split
    tiles = {p[:2] for p in run if p[1]}
    assert len(tiles) == (8 if x == "fp4" else 7) and any(p[1] == 0 for p in run)
    assert all((n, m, s, False) in run for n, m in tiles for s in (False, True))


def test_workspace_sizes_from_the_binding(L):
    from w8a8_gemm_rl_amd import binding as B

    for fn in ("qr_mxfp4_gemm", "qr_mxfp4_linear"):
        for x, fmt in (("fp4", MX4), ("fp8", MX8)):
            for shape in ((33, 512, 18944), (256, 3584, 18944), (1, 512, 256)):
                assert B.workspace_size(fn, *shape, x) == L.qr_workspace_size(fn.encode(), *shape, fmt)
        with pytest.raises(ValueError):
            B.workspace_size(fn, 16, 512, 256, "int8")
        with pytest.raises(B.QRError):
            B.workspace_size(fn, 16, 512, 200, "fp4")
    assert B.workspace_size("qr_mxfp4_gemm", 256, 3584, 18944, "fp4") > 0
    with pytest.raises(ValueError):
        B.workspace_size("qr_w8a8_gemm", 16, 512, 256, "fp4")
