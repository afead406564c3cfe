"""The 8-bit floating point calls without a GPU: the arguments they refuse (nothing is enqueued
in these tests), the struct mirrors, and the 64-bit oracle's own arithmetic."""
import ctypes
import fractions
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import fp8_oracle as O
import routing_dispatch_expert_warp_b200 as M
from routing_dispatch_expert_warp_b200 import _abi, build as B

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
P = 0x7F0000000000  # an aligned address that no refused call reads


@pytest.fixture(scope="module")
def lib():
    B.build()
    return _abi.lib()


def status(code, lib, *words):
    msg = lib.moe_last_error().decode()
    for w in words:
        assert w in msg, msg
    return code


# ------------------------------------------------------------------ the C calls
def test_quantize_rows_refuses(lib):
    def call(dtype=1, rows=4, cols=128, x=P, q=P, s=P):
        return status(lib.moe_fp8_quantize_rows(dtype, rows, cols, x, q, s, None), lib)

    assert call(rows=0, x=None, q=None, s=None) == 0
    for kw in (dict(dtype=2), dict(dtype=-1), dict(rows=-1), dict(rows=1 << 31), dict(cols=0),
               dict(cols=8), dict(cols=24), dict(cols=(1 << 24) + 16), dict(cols=-16),
               dict(x=None), dict(q=None), dict(s=None), dict(x=P + 8), dict(q=P + 4),
               dict(s=P + 2)):
        assert call(**kw) == INVALID, kw
    assert "moe_fp8_quantize_rows" in lib.moe_last_error().decode()


def test_permute_rows_refuses(lib):
    def call(d=128, T=4, x=P, a=P, q=P, s=P, **kw):
        cfg = M.make_config(T, d, 128, 8, 2, **kw)
        return lib.moe_fp8_permute_rows(ctypes.byref(cfg), x, a, q, s, None)

    for kw in (dict(d=8), dict(d=24), dict(T=0), dict(x=None), dict(a=None), dict(q=None),
               dict(s=None), dict(x=P + 8), dict(q=P + 8), dict(s=P + 8), dict(a=P + 4)):
        assert call(**kw) == INVALID, kw
    assert lib.moe_fp8_permute_rows(None, P, P, P, P, None) == INVALID


def test_quantize_weights_refuses(lib):
    def call(dtype=1, E=2, N=128, K=128, w=P, q=P, s=P):
        return lib.moe_fp8_quantize_weights(dtype, E, N, K, w, q, s, None)

    for kw in (dict(dtype=7), dict(E=0), dict(E=257), dict(N=0), dict(N=(1 << 24) + 1),
               dict(K=24), dict(K=0), dict(w=None), dict(q=None), dict(s=None), dict(w=P + 8),
               dict(q=P + 8), dict(s=P + 8)):
        assert call(**kw) == INVALID, kw


def ws_bytes(lib):
    n = ctypes.c_size_t(0)
    assert lib.moe_fp8_workspace_size(ctypes.byref(n)) == 0
    assert lib.moe_fp8_workspace_size(None) == INVALID
    return n.value


def test_workspace_refuses(lib):
    n = ws_bytes(lib)
    assert lib.moe_fp8_workspace_init(None, n, None) == INVALID
    assert lib.moe_fp8_workspace_init(P + 16, n, None) == INVALID
    assert lib.moe_fp8_workspace_init(P, n - 1, None) == WORKSPACE


def test_grouped_gemm_refuses(lib):
    n = ws_bytes(lib)

    def call(E=2, rows=4, N=128, K=128, a=P, sa=P, f=P, c=P, w=P, sw=P, o=P, ws=P, nb=n):
        return lib.moe_fp8_grouped_gemm(E, rows, N, K, a, sa, f, c, w, sw, o, ws, nb, None)

    assert call(rows=0) == 0
    for kw in (dict(E=0), dict(E=257), dict(rows=-1), dict(rows=1 << 31), dict(N=0), dict(N=4),
               dict(N=12), dict(N=(1 << 24) + 8), dict(K=0), dict(K=8), dict(K=136), dict(a=None),
               dict(sa=None), dict(f=None), dict(c=None), dict(w=None), dict(sw=None),
               dict(o=None), dict(ws=None), dict(ws=P + 128), dict(a=P + 8), dict(sa=P + 8),
               dict(w=P + 8), dict(sw=P + 8), dict(o=P + 8)):
        assert call(**kw) == INVALID, kw
    assert call(nb=n - 1) == WORKSPACE
    assert call(rows=(1 << 31) - 1, N=1 << 24) == UNSUPPORTED


def experts_struct(**kw):
    d = {name: P for name, _ in _abi.MoeFp8Experts._fields_}
    d.update(kw)
    return _abi.MoeFp8Experts(**d)


def test_expert_ffn_refuses(lib):
    n = ws_bytes(lib)

    def call(cfg=None, e=experts_struct(), x=P, xs=P, o=P, k=P, h=P, hs=P, y=P, ws=P, nb=n):
        cfg = cfg or M.make_config(4, 128, 256, 8, 2)
        return lib.moe_expert_ffn_fp8(ctypes.byref(cfg), x, xs, o, k,
                                      None if e is None else ctypes.byref(e), h, hs, y, ws, nb,
                                      None)

    for kw in (dict(cfg=M.make_config(4, 136, 256, 8, 2)), dict(cfg=M.make_config(4, 128, 132, 8, 2)),
               dict(cfg=M.make_config(4, 128, 8, 8, 2)), dict(e=None), dict(x=None), dict(xs=None),
               dict(o=None), dict(k=None), dict(h=None), dict(hs=None), dict(y=None),
               dict(ws=None), dict(ws=P + 64), dict(x=P + 8), dict(y=P + 8), dict(h=P + 8)):
        assert call(**kw) == INVALID, kw
    for name, _ in _abi.MoeFp8Experts._fields_:
        assert call(e=experts_struct(**{name: None})) == INVALID, name
        assert call(e=experts_struct(**{name: P + 8})) == INVALID, name
    assert call(nb=n - 1) == WORKSPACE
    assert call(cfg=M.make_config(4, 128, 256, 8, 2, dtype=M.F32)) == UNSUPPORTED


def test_layer_refuses(lib):
    n = ws_bytes(lib)
    cfg = M.make_config(4, 128, 256, 8, 2)
    inp, buf = _abi.MoeLayerInputs(), _abi.MoeLayerBuffers()
    for f, _ in _abi.MoeLayerBuffers._fields_:
        setattr(buf, f, P)
    e, fb = experts_struct(), _abi.MoeFp8Buffers(P, P, P, P)

    def call(cfg=cfg, i=inp, e=e, b=buf, f=fb, w=P, fw=P, fn=n):
        ref = lambda s: None if s is None else ctypes.byref(s)  # noqa: E731
        return lib.moe_layer_forward_fp8(ref(cfg), ref(i), ref(e), ref(b), ref(f), w,
                                         M.workspace_size(M.make_config(4, 128, 256, 8, 2)), fw,
                                         fn, None)

    assert call() == INVALID  # inputs without x
    for kw in (dict(cfg=None), dict(i=None), dict(e=None), dict(b=None), dict(f=None),
               dict(w=None), dict(fw=None), dict(f=_abi.MoeFp8Buffers(P, P, None, P)),
               dict(cfg=M.make_config(4, 136, 256, 8, 2))):
        assert call(**kw) == INVALID, kw
    assert call(fn=n - 1) == WORKSPACE
    assert call(cfg=M.make_config(4, 128, 256, 8, 2, dtype=M.F32)) == UNSUPPORTED


def test_layer_refuses_before_it_enqueues(lib):
    """What the expert stages would refuse is refused before the router runs: here, where no
    kernel can run, the refusal and not the failed launch is what comes back."""
    n = ws_bytes(lib)
    cfg = M.make_config(4, 128, 256, 8, 2)
    inp = _abi.MoeLayerInputs()
    inp.x = inp.w_router = P
    buf = _abi.MoeLayerBuffers()
    for f, _ in _abi.MoeLayerBuffers._fields_:
        setattr(buf, f, P)
    for e, fb in ((experts_struct(up_scale=None), (P, P, P, P)),
                  (experts_struct(w_down=P + 8), (P, P, P, P)),
                  (experts_struct(), (P + 4, P, P, P)),
                  (experts_struct(), (P, P, P, P + 8))):
        f = _abi.MoeFp8Buffers(*fb)
        assert lib.moe_layer_forward_fp8(ctypes.byref(cfg), ctypes.byref(inp), ctypes.byref(e),
                                         ctypes.byref(buf), ctypes.byref(f), P,
                                         M.workspace_size(cfg), P, n, None) == INVALID
        assert b"moe_layer_forward_fp8" in lib.moe_last_error()


def test_layer_class_refuses_what_does_not_fit(lib):
    E, d, f = 4, 64, 48
    q = lambda *s: torch.zeros(s, dtype=M.fp8.E4M3)  # noqa: E731
    z = lambda *s: torch.zeros(M.fp8_scale_shape(s))  # noqa: E731
    ex = M.Fp8Experts(q(E, f, d), z(E, f, d), q(E, f, d), z(E, f, d), q(E, d, f), z(E, d, f))
    cfg = M.make_config(4, d, f, E, 1)
    w = torch.zeros(d, E)
    for router, bias in ((w.bfloat16(), None), (w.t().contiguous(), None), (w[:, ::2], None),
                         (w, torch.zeros(E + 1)), (w, torch.zeros(3, E)), (w, torch.zeros(4, 2)),
                         (w, torch.zeros(E, dtype=torch.float64)), (w.to("meta"), None)):
        with pytest.raises(ValueError):
            M.MoELayerFp8(cfg, router, ex, bias)


def test_struct_layout_matches_header(tmp_path):
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "moe.h"\nint main(void) {\n'
                   'printf("%zu %zu %zu %zu", sizeof(moe_fp8_experts_t), sizeof(moe_fp8_buffers_t),'
                   'offsetof(moe_fp8_experts_t, down_scale), offsetof(moe_fp8_buffers_t, h_scale));'
                   'return 0; }\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", B.INCLUDE, str(src), "-o", str(exe)], check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    assert [int(v) for v in got] == [
        ctypes.sizeof(_abi.MoeFp8Experts), ctypes.sizeof(_abi.MoeFp8Buffers),
        _abi.MoeFp8Experts.down_scale.offset, _abi.MoeFp8Buffers.h_scale.offset]


# ------------------------------------------------------------------ the Python calls
def e4m3(*shape):
    return torch.zeros(shape, dtype=torch.float8_e4m3fn)


def test_python_calls_refuse_what_does_not_fit(lib):
    x, q, s = torch.zeros(4, 256), e4m3(4, 256), torch.zeros(4, 2)
    rows = M.moe_fp8_quantize_rows
    for bad in ((x.half(), q, s), (x[0], q, s), (x.t(), q, s), (x, q.float(), s),
                (x, e4m3(4, 255), s), (x, q, torch.zeros(4, 3)), (x, q, s.double()),
                (x, q, torch.zeros(2, 4).t())):
        with pytest.raises(ValueError):
            rows(*bad)
    with pytest.raises(ValueError, match="CUDA"):
        rows(x, q, s)
    w, wq, ws = torch.zeros(2, 200, 144), e4m3(2, 200, 144), torch.zeros(2, 2, 2)
    for bad in ((w[0], wq, ws), (w, wq[:1], ws), (w, wq, ws[:, :1])):
        with pytest.raises(ValueError):
            M.moe_fp8_quantize_weights(*bad)
    cfg = M.make_config(4, 256, 128, 8, 2)
    pick = torch.zeros((4, 2), dtype=torch.int32)
    xq, xs = e4m3(8, 256), torch.zeros(8, 2)
    xb = x.bfloat16()
    for bad in ((x, pick, xq, xs), (xb, pick.long(), xq, xs), (xb, pick[:3], xq, xs),
                (xb, pick, xq[:7], xs), (xb, pick, xq, xs[:, :1])):
        with pytest.raises(ValueError):
            M.moe_fp8_permute_rows(cfg, *bad)
    i32 = torch.zeros(2, dtype=torch.int32)
    ok = [e4m3(4, 144), torch.zeros(4, 2), i32, i32, wq, ws, torch.zeros((4, 200)).bfloat16(),
          torch.zeros(64, dtype=torch.uint8)]
    for at, bad in ((0, e4m3(4, 128)), (0, e4m3(4)), (1, torch.zeros(4, 1)), (2, i32.long()),
                    (2, torch.zeros(5, dtype=torch.int32)), (3, i32[:1]), (4, wq[0]),
                    (4, wq.float()), (5, torch.zeros(2, 2, 1)), (6, torch.zeros(4, 200)),
                    (6, torch.zeros((4, 208)).bfloat16()), (7, torch.zeros(64))):
        args = list(ok)
        args[at] = bad
        with pytest.raises(ValueError):
            M.moe_fp8_grouped_gemm(*args)
    with pytest.raises(ValueError, match="CUDA"):
        M.moe_fp8_grouped_gemm(*ok)


def test_experts_have_matching_halves():
    E, f, d = 2, 144, 272
    up = (e4m3(E, f, d), torch.zeros(E, 2, 3))
    down = (e4m3(E, d, f), torch.zeros(E, 3, 2))
    ex = M.Fp8Experts(*up, *up, *down)
    for bad in ((*up, *down, *down), (*up, *up, *up), (up[0], down[1], *up, *down),
                (up[0].float(), up[1], *up, *down), (*up, up[0][:1], up[1], *down),
                (*up, *up, down[0], down[1].double())):
        with pytest.raises(ValueError):
            M.Fp8Experts(*bad)
    with pytest.raises(ValueError, match="layer"):
        M.MoELayerFp8(M.make_config(4, d, f + 16, E, 1), None, ex)
    with pytest.raises(ValueError):
        M.fp8_scale_shape((3,))


# ------------------------------------------------------------------ the oracle
def test_oracle_numbers_are_torchs():
    c = torch.arange(256, dtype=torch.uint8)
    ours = O.code_values(c.numpy())
    theirs = c.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ours, theirs, equal_nan=True)


def test_oracle_rounding_is_to_nearest_even():
    g = torch.Generator().manual_seed(0)
    v = (torch.rand(20000, generator=g) - 0.5) * 2 ** (torch.rand(20000, generator=g) * 20 - 10)
    v = torch.cat([v.clamp(-448, 448), torch.from_numpy(O.BORDERS).float(),
                   -torch.from_numpy(O.BORDERS).float()])
    assert np.array_equal(O.to_codes(v.double().numpy()),
                          v.to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_bf16_quotients_keep_their_distance_from_borders():
    """448 x / m of two 8-bit significands is on a border of two e4m3 numbers or at least 2^-13
    of it away: what the conversion of bf16 entries rests on."""
    nearest = fractions.Fraction(1)
    for m in range(128, 256):
        for x in range(128, 256):
            for shift in range(-12, 1):
                q = fractions.Fraction(7 * x, m) * fractions.Fraction(2) ** (6 + shift)
                at = np.searchsorted(O.BORDERS, float(q))
                for i in (at - 1, at):
                    if 0 <= i < len(O.BORDERS):
                        b = fractions.Fraction(O.BORDERS[i])
                        if q != b:
                            nearest = min(nearest, abs(q / b - 1))
    assert nearest > fractions.Fraction(1, 2 ** 13)


def test_oracle_products_and_blocks():
    x = torch.randn(3, 272, generator=torch.Generator().manual_seed(1))
    c, s = O.quantize_rows(x)
    q = torch.from_numpy(c).view(torch.float8_e4m3fn)
    v = O.rows_value(q, torch.from_numpy(s))
    assert ((v - x.double()).abs() <= 2 ** -4 * x.double().abs() + 2 ** -10 * s.max()).all()
    w = torch.randn(1, 130, 272, generator=torch.Generator().manual_seed(2))
    c, s = O.quantize_weights(w)
    assert s.shape == (1, 2, 3)
    for n in (0, 127, 128, 129):
        for k in (0, 130, 271):
            m = w[0, n // 128 * 128:n // 128 * 128 + 128, k // 128 * 128:k // 128 * 128 + 128]
            assert s[0, n // 128, k // 128] == np.float32(m.abs().max()) / np.float32(448)


# ------------------------------------------------------------------ the largest sizes
def test_rows_that_tiles_cannot_number_are_refused(lib):
    """Rows are rounded up to whole tiles in 32 bits: 2^31 - 128 is the most that they can be."""
    n = ws_bytes(lib)

    def gemm(rows, a=P):
        return lib.moe_fp8_grouped_gemm(1, rows, 8, 16, a, P, P, P, P, P, P, P, n, None)

    for rows in range(2 ** 31 - 127, 2 ** 31):
        assert gemm(rows) == UNSUPPORTED, rows
    assert gemm(2 ** 31 - 128, a=None) == INVALID  # as far as the pointers

    def ffn(T, x=P):
        cfg = M.make_config(T, 16, 16, 1, 1)
        return lib.moe_expert_ffn_fp8(ctypes.byref(cfg), x, P, P, P, ctypes.byref(experts_struct()),
                                      P, P, P, P, n, None)

    assert ffn(2 ** 31 - 1) == ffn(2 ** 31 - 127) == UNSUPPORTED
    assert ffn(2 ** 31 - 128, x=None) == INVALID


def test_tiles_that_32_bits_cannot_number_are_refused(lib):
    """A block steps from tile to tile in 32 bits: the step past the last one must fit too."""
    n = ws_bytes(lib)

    def gemm(rows, N, a=P):
        return lib.moe_fp8_grouped_gemm(1, rows, N, 16, a, P, P, P, P, P, P, P, n, None)

    # (rows / 128 + 1) x 128 tiles of 128 x 128
    assert gemm(128 * (2 ** 24 - 2), 128 * 128) == UNSUPPORTED
    assert gemm(128 * (2 ** 24 - 1024), 128 * 128, a=None) == INVALID


# ------------------------------------------------------------------ the kernels' source
def test_a_warpgroup_has_one_register_split():
    """All warps of a warpgroup have to execute the same setmaxnreg: a kernel says it once for the
    four control warps, before they part, and once for the epilogue's."""
    seen = 0
    for name in sorted(os.listdir(B.CSRC)):
        with open(os.path.join(B.CSRC, name)) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        if "setmaxnreg" not in text:
            continue
        seen += 1
        assert text.count('("setmaxnreg.dec') == text.count('("setmaxnreg.inc') == 1, name
        assert len(re.findall(r"if \(warp < CTRL_WARPS\) \{\s*regs_dec<\w+>\(\);", text)) == 1, name
        assert len(re.findall(r"regs_dec<\w+>\(\)", text)) == 1, name
        assert len(re.findall(r"\} else \{\s*regs_inc<\w+>\(\);", text)) == 1, name
        assert len(re.findall(r"regs_inc<\w+>\(\)", text)) == 1, name
    assert seen == 1
