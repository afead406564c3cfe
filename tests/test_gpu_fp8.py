"""The 8-bit floating point operators against their definition in 64 bits: quantisation of
rows and weights bit by bit, ragged products and the SwiGLU FFN within the rounding that their
arithmetic admits, and the calls around them (streams, graphs, rows outside the buckets)."""
import numpy as np
import pytest
import torch

import fp8_oracle as O
import routing_dispatch_expert_warp_b200 as M
from routing_dispatch_expert_warp_b200 import workload as W

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    yield


def gen(seed):
    return torch.Generator().manual_seed(seed)


def codes(q):
    return q.view(torch.uint8).cpu().numpy()


def assert_same_scales(got, ref):
    got = got.cpu().numpy()
    assert got.shape == ref.shape
    assert np.array_equal(got.view(np.uint32)[~np.isnan(ref)], ref.view(np.uint32)[~np.isnan(ref)])
    assert np.isnan(got[np.isnan(ref)]).all()


def assert_same_codes(got, ref):
    got = codes(got)
    nan = (ref & 0x7F) == 0x7F
    assert np.array_equal(got[~nan], ref[~nan]), (got != ref).sum()
    assert ((got[nan] & 0x7F) == 0x7F).all()


def values(shape, dtype, seed, kind="normal"):
    g = gen(seed)
    x = torch.randn(shape, generator=g, dtype=torch.float64)
    if kind == "outliers":
        x = x * (1 + 100 * (torch.rand(shape, generator=g) < 0.01))
    elif kind == "spread":   # magnitudes over the whole range of the type
        x = x * torch.exp2(torch.rand(shape, generator=g) * 240 - 130)
    elif kind == "tiny":     # blocks below the floor, subnormals among them
        x = x * torch.exp2(torch.rand(shape, generator=g) * 60 - 150)
    elif kind == "borders":  # short fractions: quotients on the borders of e4m3
        x = torch.randint(-32, 33, shape, generator=g).double() / 8
    elif kind == "zero":
        x = torch.zeros(shape, dtype=torch.float64)
    return x.to(dtype)


# ------------------------------------------------------------------ rows
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 128), (3, 144), (7, 1520), (129, 528),
                                       (1000, 4096), (2, 16384), (1003, 16), (77, 128),
                                       (301, 176), (6, 256), (5, 272)])
@pytest.mark.parametrize("kind", ["normal", "outliers", "spread", "tiny", "borders", "zero"])
def test_rows(rows, cols, dtype, kind):
    x = values((rows, cols), dtype, rows + cols, kind)
    q = torch.empty((rows, cols), dtype=E4M3, device="cuda")
    s = torch.empty((rows, O.blocks(cols)), device="cuda")
    M.moe_fp8_quantize_rows(x.cuda(), q, s)
    ref_q, ref_s = O.quantize_rows(x)
    assert_same_scales(s, ref_s)
    assert_same_codes(q, ref_q)


def test_rows_every_bf16_quotient():
    """All pairs of significands: x / m for x, m in 128 .. 255, m the block's largest."""
    m, x = torch.meshgrid(torch.arange(128, 256), torch.arange(128, 256), indexing="ij")
    rows = torch.zeros((128 * 128, 16))
    rows[:, 0] = m.flatten().float()
    for i in range(1, 15):  # and over the exponents that reach e4m3's smallest steps
        rows[:, i] = x.flatten().float() * 2.0 ** (-1 - i) * (-1) ** i
    rows = rows.bfloat16()
    q = torch.empty(rows.shape, dtype=E4M3, device="cuda")
    s = torch.empty((rows.shape[0], 1), device="cuda")
    M.moe_fp8_quantize_rows(rows.cuda(), q, s)
    ref_q, ref_s = O.quantize_rows(rows)
    assert_same_scales(s, ref_s)
    assert_same_codes(q, ref_q)


def test_rows_fp32_next_to_borders():
    """fp32 entries at the fp32 numbers next to a border of e4m3, on both sides of it."""
    g = gen(5)
    m = (1 + torch.rand(4096, generator=g)).float()
    border = torch.from_numpy(O.BORDERS)[torch.randint(0, 126, (4096, 15), generator=g)]
    x = (border * m[:, None].double() / 448).float()
    step = torch.randint(-2, 3, x.shape, generator=g, dtype=torch.int32)
    x = (x.view(torch.int32) + step).view(torch.float32)
    rows = torch.cat([m[:, None], x], 1)
    q = torch.empty(rows.shape, dtype=E4M3, device="cuda")
    s = torch.empty((rows.shape[0], 1), device="cuda")
    M.moe_fp8_quantize_rows(rows.cuda(), q, s)
    ref_q, ref_s = O.quantize_rows(rows)
    assert_same_scales(s, ref_s)
    assert_same_codes(q, ref_q)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_rows_with_nan_and_infinity(dtype):
    x = values((6, 400), dtype, 3)
    x[0, 5] = float("nan")
    x[1, 130] = float("inf")
    x[2, 399] = -float("inf")
    x[3, 128] = float("nan")
    x[3, 129] = float("inf")
    q = torch.empty(x.shape, dtype=E4M3, device="cuda")
    s = torch.empty((6, 4), device="cuda")
    M.moe_fp8_quantize_rows(x.cuda(), q, s)
    ref_q, ref_s = O.quantize_rows(x)
    assert np.isnan(ref_s).sum() == 4
    assert_same_scales(s, ref_s)
    assert_same_codes(q, ref_q)


def test_no_rows():
    q = torch.empty((0, 128), dtype=E4M3, device="cuda")
    M.moe_fp8_quantize_rows(torch.empty((0, 128), device="cuda"), q,
                            torch.empty((0, 1), device="cuda"))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,d,E,k,cf", [(1, 16, 1, 1, 0.0), (1, 4096, 8, 2, 0.0),
                                        (37, 1520, 13, 8, 0.5), (600, 656, 256, 8, 1.0),
                                        (64, 7168, 4, 3, 0.0), (203, 32, 16, 8, 0.7),
                                (50, 128, 8, 5, 0.0), (77, 240, 8, 2, 0.6)])
def test_permute_writes_the_kept_picks_rows(T, d, E, k, cf, dtype):
    g = gen(T + d)
    cfg = M.make_config(T, d, 128, E, k, capacity_factor=cf,
                        dtype=M.F32 if dtype == torch.float32 else M.BF16)
    R = M.max_rows(cfg)
    x = values((T, d), dtype, T)
    row = torch.full((T * k,), -1, dtype=torch.int32)
    kept = torch.randperm(T * k, generator=g)[:max(1, min(R - 1, T * k))]
    row[kept] = torch.randperm(R, generator=g)[:len(kept)].int()
    row = row.view(T, k)
    q = torch.full((R, d), 0.5, device="cuda").to(E4M3)
    s = torch.full((R, O.blocks(d)), 7.0, device="cuda")
    M.moe_fp8_permute_rows(cfg, x.cuda(), row.cuda(), q, s)
    tq, ts = O.quantize_rows(x)
    ref_q = np.full((R, d), 0x30, dtype=np.uint8)
    ref_s = np.full((R, O.blocks(d)), 7.0, dtype=np.float32)
    for t in range(T):
        for r in row[t].tolist():
            if r >= 0:
                ref_q[r], ref_s[r] = tq[t], ts[t]
    assert_same_scales(s, ref_s)
    assert_same_codes(q, ref_q)


def test_permute_skips_rows_outside_the_buffer():
    cfg = M.make_config(4, 128, 128, 2, 2)
    row = torch.tensor([[0, 8], [1 << 30, 1], [-5, 2], [7, -1]], dtype=torch.int32)
    full = torch.zeros((12, 128), device="cuda").to(E4M3)
    scale = torch.zeros((12, 1), device="cuda")
    M.moe_fp8_permute_rows(cfg, torch.ones((4, 128), device="cuda").bfloat16(), row.cuda(),
                           full[2:10], scale.narrow(0, 4, 8))
    wrote = [i for i in range(12) if codes(full)[i].any()]
    assert wrote == [2, 3, 4, 9]
    assert (scale != 0).flatten().nonzero().flatten().tolist() == [4, 5, 6, 11]


# ------------------------------------------------------------------ weights
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 1, 16), (2, 128, 128), (3, 200, 272), (5, 129, 144),
                                   (1, 1000, 1520), (256, 8, 16)])
@pytest.mark.parametrize("kind", ["normal", "spread", "borders"])
def test_weights(shape, dtype, kind):
    w = values(shape, dtype, sum(shape), kind)
    q = torch.empty(shape, dtype=E4M3, device="cuda")
    s = torch.empty(M.fp8_scale_shape(shape), device="cuda")
    M.moe_fp8_quantize_weights(w.cuda(), q, s)
    ref_q, ref_s = O.quantize_weights(w)
    assert_same_scales(s, ref_s)
    assert_same_codes(q, ref_q)


def test_weights_with_nan():
    w = values((2, 260, 272), torch.bfloat16, 1)
    w[1, 129, 271] = float("nan")
    w[0, 0, 0] = float("inf")
    q = torch.empty(w.shape, dtype=E4M3, device="cuda")
    s = torch.empty(M.fp8_scale_shape(w.shape), device="cuda")
    M.moe_fp8_quantize_weights(w.cuda(), q, s)
    ref_q, ref_s = O.quantize_weights(w)
    assert np.isnan(ref_s).sum() == 2
    assert_same_scales(s, ref_s)
    assert_same_codes(q, ref_q)


# ------------------------------------------------------------------ products
def quantized_rows(x):
    q = torch.empty(x.shape, dtype=E4M3, device="cuda")
    s = torch.empty(M.fp8_scale_shape(x.shape), device="cuda")
    M.moe_fp8_quantize_rows(x.cuda(), q, s)
    return q, s


def quantized_weights(w):
    q = torch.empty(w.shape, dtype=E4M3, device="cuda")
    s = torch.empty(M.fp8_scale_shape(w.shape), device="cuda")
    M.moe_fp8_quantize_weights(w.cuda(), q, s)
    return q, s


def starts(counts, gap=0):
    at, first = 0, []
    for c in counts:
        first.append(at)
        at += c + gap
    return first, at


GEMM = [  # counts, N, K
    ([1], 8, 16),
    ([1], 256, 128),
    ([2, 0, 1], 136, 144),
    ([128], 256, 256),
    ([129, 127], 264, 272),
    ([0, 0, 300, 0, 31, 33, 64, 96, 97], 1000, 1520),
    ([64] * 3, 4096, 7168),
    ([700, 5], 520, 2048),
    ([1] * 256, 128, 128),
    ([3, 0] * 128, 48, 400),
    ([2000], 640, 128),
    ([0, 0], 256, 256),
    ([1, 1], 4096, 14336),
    ([260, 513, 1, 255, 256, 257], 768, 640),
    ([200, 0, 0, 1, 0, 0, 17, 0], 1000, 1520),   # one long bucket among few rows
    ([64, 16, 15, 17, 48, 49, 63, 65, 0, 1, 0, 2], 520, 272),
    ([5], 14336, 4096),
    ([4] * 32, 7168, 2048),    # seven rounds of tiles on 148 SMs, the last one nearly empty
    ([1, 30, 2, 0, 9], 30000, 1040),
]


@pytest.mark.parametrize("gap", [0, 3])
@pytest.mark.parametrize("counts,N,K", GEMM)
def test_grouped_gemm(counts, N, K, gap):
    g = gen(N + K)
    E = len(counts)
    first, rows = starts(counts, gap)
    rows += 2  # rows behind the last bucket
    a_q, a_s = quantized_rows(torch.randn((rows, K), generator=g).bfloat16())
    w_q, w_s = quantized_weights(torch.randn((E, N, K), generator=g) / K ** 0.5)
    out = torch.full((rows, N), 3.25, dtype=torch.bfloat16, device="cuda")
    ws = M.alloc_fp8_workspace()
    i32 = dict(dtype=torch.int32, device="cuda")
    M.moe_fp8_grouped_gemm(a_q, a_s, torch.tensor(first, **i32), torch.tensor(counts, **i32),
                           w_q, w_s, out, ws)
    M.moe_check_device_error(ws)
    check_product(out, a_q, a_s, w_q, w_s, first, counts)


def check_product(out, a_q, a_s, w_q, w_s, first, counts, untouched=3.25):
    got = out.cpu().double()
    a = O.rows_value(a_q, a_s)
    seen = torch.zeros(len(got), dtype=torch.bool)
    tol = O.sum_error(a.shape[1])
    for e, (r0, c) in enumerate(zip(first, counts)):
        if c == 0:
            continue
        at = slice(r0, r0 + c)
        ref, mag = O.product(a[at], O.weight_value(w_q[e], w_s[e]))
        room = O.BF16_HALF_STEP * ref.abs() + (1 + O.BF16_HALF_STEP) * tol * mag
        assert ((got[at] - ref).abs() <= room).all(), (e, (got[at] - ref).abs().max())
        seen[at] = True
    assert (got[~seen] == untouched).all()


def test_grouped_gemm_equal_calls_give_equal_bits_and_streams_do_not_matter():
    counts, N, K = [5, 0, 130, 1], 1000, 2064
    first, rows = starts(counts)
    g = gen(1)
    a_q, a_s = quantized_rows(torch.randn((rows, K), generator=g))
    w_q, w_s = quantized_weights(torch.randn((4, N, K), generator=g))
    i32 = dict(dtype=torch.int32, device="cuda")
    f, c = torch.tensor(first, **i32), torch.tensor(counts, **i32)
    outs = []
    torch.cuda.synchronize()
    for stream in (None, None, torch.cuda.Stream(), torch.cuda.Stream()):
        out = torch.zeros((rows, N), dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        ws = M.alloc_fp8_workspace(stream=stream)
        for _ in range(3):
            M.moe_fp8_grouped_gemm(a_q, a_s, f, c, w_q, w_s, out, ws, stream)
        outs.append(out)
    torch.cuda.synchronize()
    for out in outs[1:]:
        assert torch.equal(out, outs[0])


def test_grouped_gemm_nan_stays_in_its_row():
    K, N = 384, 256
    x = torch.randn((70, K), generator=gen(2))
    x[33, 200] = float("nan")
    a_q, a_s = quantized_rows(x)
    w_q, w_s = quantized_weights(torch.randn((1, N, K), generator=gen(3)))
    i32 = dict(dtype=torch.int32, device="cuda")
    out = torch.zeros((70, N), dtype=torch.bfloat16, device="cuda")
    M.moe_fp8_grouped_gemm(a_q, a_s, torch.zeros(1, **i32), torch.full((1,), 70, **i32), w_q,
                           w_s, out, M.alloc_fp8_workspace())
    nan = out.isnan().cpu()
    assert nan[33].all() and nan.sum() == N


def test_grouped_gemm_reports_a_bucket_outside_the_rows():
    K, N, rows = 128, 256, 40
    a_q, a_s = quantized_rows(torch.randn((rows, K), generator=gen(2)))
    w_q, w_s = quantized_weights(torch.randn((4, N, K), generator=gen(3)))
    i32 = dict(dtype=torch.int32, device="cuda")
    first, counts = [0, 30, -3, 10], [10, 11, 2, 20]
    out = torch.full((rows, N), 3.25, dtype=torch.bfloat16, device="cuda")
    ws = M.alloc_fp8_workspace()
    M.moe_fp8_grouped_gemm(a_q, a_s, torch.tensor(first, **i32), torch.tensor(counts, **i32),
                           w_q, w_s, out, ws)
    with pytest.raises(M.MoEError) as e:
        M.moe_check_device_error(ws)
    assert e.value.status == 6 and "bucket" in str(e.value)
    M.moe_check_device_error(ws)  # read once
    check_product(out, a_q, a_s, w_q, w_s, [0, 0, 0, 10], [10, 0, 0, 20])


@pytest.mark.parametrize("seed", range(24))
def test_grouped_gemm_random_buckets(seed):
    """Random sizes and buckets, few rows and many; the workspace is used again and again, as the
    pieces of cut tiles need it."""
    g = np.random.default_rng(seed)
    E = int(g.choice([1, 2, 5, 16, 64, 256]))
    K, N = 16 * int(g.integers(1, 160)), 8 * int(g.integers(1, 200))
    mean = float(g.choice([0.3, 3, 20, 100])) if E <= 16 else float(g.choice([0.3, 3]))
    ws = M.alloc_fp8_workspace()
    w_q, w_s = quantized_weights(torch.randn((E, N, K), generator=gen(seed)) / K ** 0.5)
    for call in range(2):
        counts = g.poisson(mean * g.exponential(1.0, E)).tolist()
        counts[int(g.integers(E))] += 1
        first, rows = starts(counts, int(g.integers(0, 3)))
        a_q, a_s = quantized_rows(torch.randn((rows, K), generator=gen(seed + 50)).bfloat16())
        out = torch.full((rows, N), 3.25, dtype=torch.bfloat16, device="cuda")
        i32 = dict(dtype=torch.int32, device="cuda")
        f, c = torch.tensor(first, **i32), torch.tensor(counts, **i32)
        M.moe_fp8_grouped_gemm(a_q, a_s, f, c, w_q, w_s, out, ws)
        M.moe_check_device_error(ws)
        check_product(out, a_q, a_s, w_q, w_s, first, counts)
        again = torch.full((rows, N), 3.25, dtype=torch.bfloat16, device="cuda")
        M.moe_fp8_grouped_gemm(a_q, a_s, f, c, w_q, w_s, again, ws)
        assert torch.equal(out, again)


def test_grouped_gemm_buckets_in_any_order():
    """Buckets need not lie in the experts' order, nor start where another ends."""
    first, counts, rows, N, K = [90, 0, 40, 10], [9, 7, 33, 20], 100, 264, 400
    a_q, a_s = quantized_rows(torch.randn((rows, K), generator=gen(1)))
    w_q, w_s = quantized_weights(torch.randn((4, N, K), generator=gen(2)))
    i32 = dict(dtype=torch.int32, device="cuda")
    out = torch.full((rows, N), 3.25, dtype=torch.bfloat16, device="cuda")
    ws = M.alloc_fp8_workspace()
    M.moe_fp8_grouped_gemm(a_q, a_s, torch.tensor(first, **i32), torch.tensor(counts, **i32),
                           w_q, w_s, out, ws)
    M.moe_check_device_error(ws)
    check_product(out, a_q, a_s, w_q, w_s, first, counts)


@pytest.mark.parametrize("E,rows,N", [(1, 600000, 4096), (256, 8000, 272000)],
                         ids=["many rows", "few rows"])
def test_grouped_gemm_offsets_beyond_32_bits(E, rows, N):
    """The last rows' offsets in the output pass 2^31 elements, in either kernel."""
    K, last = 16, slice(rows - 3, rows)
    counts = [rows] if E == 1 else [0] * (E - 1) + [3]
    first = [0] * (E - 1) + [rows - counts[-1]]
    g = gen(4)
    a_q, a_s = quantized_rows(torch.randn((1000, K), generator=g).repeat(rows // 1000, 1))
    w = torch.zeros((E, N, K), device="cuda")
    w[-1] = torch.randn((N, K), generator=g).cuda()
    w_q, w_s = quantized_weights(w)
    out = torch.full((rows, N), 3.25, dtype=torch.bfloat16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    ws = M.alloc_fp8_workspace()
    M.moe_fp8_grouped_gemm(a_q, a_s, torch.tensor(first, **i32), torch.tensor(counts, **i32),
                           w_q, w_s, out, ws)
    M.moe_check_device_error(ws)
    check_product(out[last], a_q[last], a_s[last], w_q[-1:], w_s[-1:], [0], [3])
    assert E == 1 or (out[-4] == 3.25).all()


def test_rows_offsets_beyond_32_bits():
    rows, cols = 140000, 16384
    x = torch.randn((7, cols), generator=gen(6)).bfloat16()
    big = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    big[-7:] = x.cuda()
    q = torch.empty((rows, cols), dtype=E4M3, device="cuda")
    s = torch.empty((rows, O.blocks(cols)), device="cuda")
    M.moe_fp8_quantize_rows(big, q, s)
    ref_q, ref_s = O.quantize_rows(x)
    assert_same_scales(s[-7:], ref_s)
    assert_same_codes(q[-7:], ref_q)
    assert not q[:-7].view(torch.uint8)[::1000].any()


def test_misaligned_tensors_are_refused():
    x = torch.zeros((4, 256), device="cuda").bfloat16()
    q = torch.zeros((4, 256), device="cuda").to(E4M3)
    s = torch.zeros((9,), device="cuda")[1:].view(4, 2)
    with pytest.raises(M.MoEError) as e:
        M.moe_fp8_quantize_rows(x, q, s)
    assert e.value.status == 1 and "aligned" in str(e.value)


def test_nothing_is_written_outside_the_outputs():
    """Every output inside a larger allocation whose other bytes hold a pattern."""
    blocks = []

    def inside(shape, dtype):
        n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
        full = torch.full((1024 + n + 1024,), 0xA5, dtype=torch.uint8, device="cuda")
        blocks.append((full, n))
        return full[1024:1024 + n].view(dtype).view(shape)

    for counts, d, f in (([1, 0, 37, 2], 272, 400), ([200, 3, 150], 400, 272)):
        E, rows = len(counts), sum(counts)
        first, _ = starts(counts)
        i32 = dict(dtype=torch.int32, device="cuda")
        cfg = M.make_config(rows, d, f, E, 1)
        x = torch.randn((rows, d), generator=gen(1)).cuda().bfloat16()
        x_q, x_s = inside((rows, d), E4M3), inside((rows, O.blocks(d)), torch.float32)
        M.moe_fp8_permute_rows(cfg, x, torch.arange(rows, **i32).view(rows, 1), x_q, x_s)
        parts = []
        for shape in ((E, f, d), (E, f, d), (E, d, f)):
            w = torch.randn(shape, generator=gen(2)).cuda()
            parts += [inside(shape, E4M3), inside(M.fp8_scale_shape(shape), torch.float32)]
            M.moe_fp8_quantize_weights(w, *parts[-2:])
        h_q, h_s = inside((rows, f), E4M3), inside((rows, O.blocks(f)), torch.float32)
        y = inside((rows, d), torch.bfloat16)
        ws = inside((M.fp8_workspace_size(),), torch.uint8)
        M.moe_fp8_workspace_init(ws)
        M.moe_expert_ffn_fp8(cfg, x_q, x_s, torch.tensor(first, **i32),
                             torch.tensor(counts, **i32), M.Fp8Experts(*parts), h_q, h_s, y, ws)
        M.moe_check_device_error(ws)
        check_product(y, h_q, h_s, parts[4], parts[5], first, counts)
    for full, n in blocks:
        assert (full[:1024] == 0xA5).all() and (full[1024 + n:] == 0xA5).all()


# ------------------------------------------------------------------ FFN
FFN = [  # counts, d, f
    ([1], 16, 16),
    ([1, 0, 1], 256, 128),
    ([130, 1, 0, 64], 272, 400),
    ([300], 1520, 720),
    ([1] * 40, 384, 144),
    ([33, 0, 257, 129], 640, 1008),
    ([2, 3], 4096, 1024),
    ([200, 0, 0, 1, 0, 0, 17, 0], 272, 400),
    ([2, 0, 0, 0, 1, 0], 1520, 2064),
    ([1], 4096, 14336),
]


def make_ffn(counts, d, f, seed=0, rows=None):
    g = gen(seed)
    E = len(counts)
    first, used = starts(counts)
    rows = used if rows is None else rows
    cfg = M.make_config(rows, d, f, E, 1)
    x_q, x_s = quantized_rows(torch.randn((rows, d), generator=g).bfloat16())
    experts = M.Fp8Experts.quantize(
        *(torch.randn(s, generator=g).cuda() / s[2] ** 0.5
          for s in ((E, f, d), (E, f, d), (E, d, f))))
    i32 = dict(dtype=torch.int32, device="cuda")
    offs = torch.tensor(first + [used], **i32)
    kept = torch.tensor(counts, **i32)
    h_q = torch.full((rows, f), 0.5, device="cuda").to(E4M3)
    h_s = torch.full((rows, O.blocks(f)), 7.0, device="cuda")
    y = torch.full((rows, d), 3.25, dtype=torch.bfloat16, device="cuda")
    return cfg, x_q, x_s, offs, kept, experts, h_q, h_s, y, first


@pytest.mark.parametrize("counts,d,f", FFN)
def test_ffn(counts, d, f):
    cfg, x_q, x_s, offs, kept, experts, h_q, h_s, y, first = make_ffn(
        counts, d, f, rows=sum(counts) + 3)
    ws = M.alloc_fp8_workspace()
    M.moe_expert_ffn_fp8(cfg, x_q, x_s, offs, kept, experts, h_q, h_s, y, ws)
    M.moe_check_device_error(ws)
    # the down product of the hidden rows that the kernel wrote
    check_product(y, h_q, h_s, experts.w_down, experts.down_scale, first, counts)
    # the hidden rows
    x, h = O.rows_value(x_q, x_s), O.rows_value(h_q, h_s)
    tol = O.sum_error(d)
    for e, (r0, c) in enumerate(zip(first, counts)):
        if c == 0:
            continue
        at = slice(r0, r0 + c)
        gate, gm = O.product(x[at], O.weight_value(experts.w_gate[e], experts.gate_scale[e]))
        up, um = O.product(x[at], O.weight_value(experts.w_up[e], experts.up_scale[e]))
        act = gate * torch.sigmoid(gate)
        ref = act * up
        # |silu'| < 1.1; exp, the two additions, divisions and products of silu and of the
        # quantisation: within 32 steps of fp32
        room = tol * (1.1 * gm * up.abs() + um * act.abs()) + 1.1 * tol * tol * gm * um
        room = room + 32 * 2.0 ** -24 * ref.abs()
        # the block's scale is 1 / 448 of its largest magnitude: a quotient is off by half a
        # step, at most 2^-4 of itself or 2^-10 in the smallest steps
        pad = O.blocks(f) * O.BLOCK - f
        big = torch.nn.functional.pad(ref.abs() + room, (0, pad)).unflatten(
            1, (-1, O.BLOCK)).amax(2).repeat_interleave(O.BLOCK, 1)[:, :f]
        step = torch.maximum(O.E4M3_HALF_STEP * (ref.abs() + room), 2.0 ** -10 * big / 448)
        assert ((h[at] - ref).abs() <= (1 + 2.0 ** -20) * (step + room)).all(), e
        s_ref = big[:, ::O.BLOCK] / 448
        off = (h_s[at].cpu().double() - s_ref).abs()
        rb = torch.nn.functional.pad(room, (0, pad)).unflatten(1, (-1, O.BLOCK)).amax(2)
        assert (off <= 2 * rb / 448 + 2.0 ** -23 * s_ref).all(), e
    for t, v in ((h_q.float(), 0.5), (h_s, 7.0)):
        assert (t[sum(counts):] == v).all()


def test_ffn_empty_hidden_row_is_zero():
    """A zero row gives h = 0 (scale 2^-100 / 448) and y = 0; other rows are as without it."""
    cfg, x_q, x_s, offs, kept, experts, h_q, h_s, y, _ = make_ffn([5, 4], 272, 144)
    x_q.view(torch.uint8)[2] = 0
    M.moe_expert_ffn_fp8(cfg, x_q, x_s, offs, kept, experts, h_q, h_s, y, M.alloc_fp8_workspace())
    assert (h_q.float()[2] == 0).all() and (y[2] == 0).all()
    assert (h_s[2].double() == np.float32(2.0 ** -100) / np.float32(448)).all()
    assert torch.isfinite(y).all() and (y[1] != 0).any() and (y[3] != 0).any()


def test_ffn_nan_row_stays_in_its_row():
    cfg, x_q, x_s, offs, kept, experts, h_q, h_s, y, _ = make_ffn([40, 60], 272, 400)
    x_q.view(torch.uint8)[41, 7] = 0x7F
    M.moe_expert_ffn_fp8(cfg, x_q, x_s, offs, kept, experts, h_q, h_s, y, M.alloc_fp8_workspace())
    nan = y.isnan().cpu()
    assert nan[41].all() and nan.sum() == 272 and h_s[41].isnan().all()


# ------------------------------------------------------------------ the layer
LAYERS = [
    W.reduced(W.MIXTRAL_8X7B, 300, 256, 384, capacity_factor=1.25),
    W.reduced(W.DSV3_PREFILL_ZIPF, 600, 256, 128, capacity_factor=0.8, n_groups=8, topk_groups=4,
              bias_mode=1, drop_policy=2),
    W.reduced(W.MIXTRAL_8X22B_MIXED, 500, 272, 144, n_decode_tokens=8, layout=W.LAYOUT_PADDED),
    W.reduced(W.MIXTRAL_8X7B, 1, 256, 128),
]


@pytest.mark.parametrize("shape", LAYERS, ids=lambda s: s.name)
def test_layer(shape):
    """The whole layer equals its stages called one by one, its routing and statistics equal
    the bf16 layer's, and its products are right for the rows that dispatch kept."""
    inp = W.make_inputs(shape, device="cuda")
    cfg = M.config_from_shape(shape)
    experts = M.Fp8Experts.quantize(inp.w_gate, inp.w_up, inp.w_down)
    layer = M.MoELayerFp8(cfg, inp.w_router, experts, inp.logit_bias)
    out = layer(inp.x).clone()
    layer.check_device_error()
    b, fb = layer.bufs, layer.fp8_bufs
    # routing, dispatch and statistics as a bf16 layer's
    ref = M.LayerBuffers.allocate(cfg)
    ws = M.alloc_workspace(cfg)
    M.moe_route(cfg, inp.x, inp.w_router, inp.logit_bias, ref.logits, ref.topk_idx, ref.topk_w, ws)
    M.moe_dispatch_scored(cfg, inp.x, ref.topk_idx, ref.logits, inp.logit_bias,
                          ref.routed_counts, ref.kept_counts, ref.expert_offsets, ref.assign_row,
                          ref.token_of_row, None, ws)
    for name in ("topk_idx", "topk_w", "routed_counts", "kept_counts", "expert_offsets",
                 "assign_row"):
        assert torch.equal(getattr(b, name), getattr(ref, name)), name
    stats = M.stats_buffer()
    assert M.moe_load_stats(cfg, ref.routed_counts, ref.kept_counts, ref.assign_row,
                            stats) == b.stats_dict()
    # the stages
    s = M.Fp8LayerBuffers.allocate(cfg)
    for t in (s.x_q, s.h_q):
        t.view(torch.uint8).fill_(0x11)
    s.layer.y_perm.fill_(3.25)
    M.moe_fp8_permute_rows(cfg, inp.x, ref.assign_row, s.x_q, s.x_scale)
    fws = M.alloc_fp8_workspace()
    M.moe_expert_ffn_fp8(cfg, s.x_q, s.x_scale, ref.expert_offsets, ref.kept_counts, experts,
                         s.h_q, s.h_scale, s.layer.y_perm, fws)
    M.moe_combine(cfg, s.layer.y_perm, ref.assign_row, ref.topk_w, s.layer.out)
    assert torch.equal(s.layer.out, out)
    first = ref.expert_offsets[:-1].tolist()
    counts = ref.kept_counts.tolist()
    tq, _ = O.quantize_rows(inp.x.cpu())
    token = ref.token_of_row.tolist()
    for r0, c in zip(first, counts):
        for r in range(r0, r0 + c):
            assert np.array_equal(codes(s.x_q)[r], tq[token[r]])
    check_product(s.layer.y_perm, s.h_q, s.h_scale, experts.w_down, experts.down_scale, first,
                  counts)
    assert torch.equal(layer(inp.x), out)


def test_layer_is_near_the_bf16_layer():
    """Six roundings to e4m3 meet in an output (x twice, gate, up, h, down): each off by at most
    2^-4 of its entry, independent over hundreds of terms, so the outputs' norm is off by less
    than sqrt(6) x 2^-4."""
    shape = W.reduced(W.MIXTRAL_8X7B, 256, 512, 640)
    inp = W.make_inputs(shape, device="cuda")
    cfg = M.config_from_shape(shape)
    a = M.MoELayer(cfg, inp.w_router, inp.w_gate, inp.w_up, inp.w_down, inp.logit_bias)(inp.x)
    experts = M.Fp8Experts.quantize(inp.w_gate, inp.w_up, inp.w_down)
    b = M.MoELayerFp8(cfg, inp.w_router, experts, inp.logit_bias)(inp.x)
    off = (a.double() - b.double()).norm() / a.double().norm()
    assert 0 < off < 6 ** 0.5 / 16


def test_layer_captured_into_a_graph():
    shape = W.reduced(W.DSV3_DECODE, 64, 256, 128)
    inp = W.make_inputs(shape, device="cuda")
    cfg = M.config_from_shape(shape)
    experts = M.Fp8Experts.quantize(inp.w_gate, inp.w_up, inp.w_down)
    layer = M.MoELayerFp8(cfg, inp.w_router, experts, inp.logit_bias)
    x = inp.x.clone()
    layer(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        layer(x, side)
    other = M.MoELayerFp8(cfg, inp.w_router, experts, inp.logit_bias)
    for seed in range(3):
        new = W.make_inputs(shape.replace(seed=seed + 50), device="cuda", weights=False).x
        x.copy_(new)
        graph.replay()
        got = layer.bufs.out.clone()
        assert torch.equal(got, other(new))
    layer.check_device_error()


@pytest.mark.parametrize("rows", [3, 300], ids=["few", "many"])
def test_calls_wait_for_whatever_came_before(rows):
    """Launches may start while the one before is ending.  Their inputs come late here from a
    kernel, a copy from the host and a memset, eagerly and captured, on their stream and from
    another one that it waits for."""
    E, N, K = 2, 520, 1040
    x = torch.randn((rows, K), generator=gen(7)).bfloat16()
    w = torch.randn((E, N, K), generator=gen(8)) / K ** 0.5
    counts = [rows - 1, 1]
    ref_q, ref_s = quantized_rows(x)
    w_q, w_s = quantized_weights(w)
    i32 = dict(dtype=torch.int32, device="cuda")
    first, count = torch.tensor([0, rows - 1], **i32), torch.tensor(counts, **i32)
    ws = M.alloc_fp8_workspace()
    want = torch.empty((rows, N), dtype=torch.bfloat16, device="cuda")
    M.moe_fp8_grouped_gemm(ref_q, ref_s, first, count, w_q, w_s, want, ws)
    check_product(want, ref_q, ref_s, w_q, w_s, [0, rows - 1], counts)
    host, host_count = x.pin_memory(), torch.tensor(counts, dtype=torch.int32).pin_memory()
    dx, dw = torch.empty_like(x, device="cuda"), w.cuda()
    q, s = torch.empty_like(ref_q), torch.empty_like(ref_s)
    wq, wsc = torch.empty_like(w_q), torch.empty_like(w_s)
    out, dcount = torch.empty_like(want), torch.empty_like(count)
    other = torch.cuda.Stream()

    def step():
        for t in (dx, s, wsc):
            t.fill_(float("nan"))
        torch.cuda._sleep(200_000)
        dx.copy_(host, non_blocking=True)
        M.moe_fp8_quantize_rows(dx, q, s)
        torch.cuda._sleep(200_000)
        here = torch.cuda.current_stream()
        other.wait_stream(here)
        with torch.cuda.stream(other):
            torch.cuda._sleep(200_000)
            M.moe_fp8_quantize_weights(dw, wq, wsc)
        here.wait_stream(other)
        dcount.zero_()
        dcount.copy_(host_count, non_blocking=True)
        M.moe_fp8_grouped_gemm(q, s, first, dcount, wq, wsc, out, ws)

    def check():
        torch.cuda.synchronize()
        M.moe_check_device_error(ws)
        assert torch.equal(out, want)
        out.fill_(0)
        for t in (q, wq):
            t.view(torch.uint8).fill_(0x7F)
        dcount.fill_(0)

    side = torch.cuda.Stream()
    for stream in (torch.cuda.current_stream(), side):
        with torch.cuda.stream(stream):
            step()
        check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for _ in range(3):
        graph.replay()
        check()


def test_layer_is_a_layer():
    """What MoELayer offers beside forward: a router weight changed in place, the counters of
    second choices, a captured forward."""
    shape = W.reduced(W.DSV3_DECODE, 64, 256, 128)
    inp = W.make_inputs(shape, device="cuda")
    cfg = M.config_from_shape(shape)
    experts = M.Fp8Experts.quantize(inp.w_gate, inp.w_up, inp.w_down)
    w_router = inp.w_router.clone()
    layer = M.MoELayerFp8(cfg, w_router, experts, inp.logit_bias)
    layer(inp.x)
    w_router.copy_(inp.w_router.flip(1))
    layer.resplit_router()
    out = layer(inp.x).clone()
    fresh = M.MoELayerFp8(cfg, w_router, experts, inp.logit_bias)
    assert torch.equal(out, fresh(inp.x))
    routed, kept, _ = layer.pick_rank_counts()
    assert torch.equal(routed.sum(0), layer.bufs.routed_counts)
    assert torch.equal(kept.sum(0), layer.bufs.kept_counts)
    x = inp.x.clone()
    graph = layer.capture(x)
    x.copy_(inp.x.flip(0))
    graph.replay()
    assert torch.equal(layer.bufs.out, fresh(inp.x.flip(0).contiguous()))
    layer.check_device_error()


def test_weights_and_workspace_on_another_stream():
    """Quantised and initialised on a side stream that runs late, into memory that the current
    stream has just let go of while still writing to it."""
    w = torch.randn(3, 256, 512, device="cuda", dtype=torch.bfloat16)
    want = M.Fp8Experts.quantize(w, w, w.transpose(1, 2).contiguous())
    wd = w.transpose(1, 2).contiguous()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for handle in (side, side.cuda_stream):
        junk = [torch.empty(w.shape, dtype=M.fp8.E4M3, device="cuda") for _ in range(6)]
        torch.cuda._sleep(20_000_000)
        for t in junk:
            t.view(torch.uint8).fill_(0x5A)
        del junk, t
        got = M.Fp8Experts.quantize(w, w, wd, handle)
        ws = M.alloc_fp8_workspace(stream=handle)
        torch.cuda.synchronize()
        for name in ("w_gate", "w_up", "w_down"):
            assert np.array_equal(codes(getattr(got, name)), codes(getattr(want, name))), name
        assert not ws[:4096].any()


def test_check_after_a_wait_ran_out_restores_the_workspace():
    """A launch that gave up leaves arrival counters behind; the layer's check reports it and
    leaves a workspace that the next forward can use."""
    shape = W.reduced(W.MIXTRAL_8X7B, 1, 1024, 512)
    inp = W.make_inputs(shape, device="cuda")
    cfg = M.config_from_shape(shape)
    experts = M.Fp8Experts.quantize(inp.w_gate, inp.w_up, inp.w_down)
    layer = M.MoELayerFp8(cfg, inp.w_router, experts, inp.logit_bias)
    want = layer(inp.x).clone()
    layer.check_device_error()
    words = layer.fp8_ws[:4096].view(torch.int32)
    assert not words.any()
    words[64:128] = 1  # counters of cut tiles
    words[0] = 1       # a status: some wait ran out
    with pytest.raises(M.MoEError):
        layer.check_device_error()
    assert not words.any()
    assert torch.equal(layer(inp.x), want)
    layer.check_device_error()


@pytest.mark.parametrize("counts", [[1, 0, 2], [150, 0, 200]], ids=["few", "many"])
def test_two_ffn_graphs_beside_each_other(counts):
    """Two captured FFNs, each with a workspace of its own, replayed on two streams at once."""
    d, f = 1520, 2064
    runs = []
    for seed in (1, 2):
        args = list(make_ffn(counts, d, f, seed))
        first = args.pop()
        ws = M.alloc_fp8_workspace()
        M.moe_expert_ffn_fp8(*args, ws)
        want = args[8].clone()
        graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            M.moe_expert_ffn_fp8(*args, ws, stream)
        args[8].zero_()
        runs.append((graph, stream, args, ws, want))
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, stream, *_ in runs:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for graph, stream, args, ws, want in runs:
        M.moe_check_device_error(ws)
        assert torch.equal(args[8], want)


@pytest.mark.parametrize("layer_code,code", [(1, 1), (1, 4), (0, 4)],
                         ids=["both ran out", "bad bucket in both", "bad bucket alone"])
def test_check_restores_the_workspace_whatever_the_errors(layer_code, code):
    """Counters of cut tiles left behind, with an error of the layer's own workspace beside the
    products', or with a bad bucket recorded before the wait that ran out."""
    shape = W.reduced(W.MIXTRAL_8X7B, 1, 1024, 512)
    inp = W.make_inputs(shape, device="cuda")
    cfg = M.config_from_shape(shape)
    experts = M.Fp8Experts.quantize(inp.w_gate, inp.w_up, inp.w_down)
    layer = M.MoELayerFp8(cfg, inp.w_router, experts, inp.logit_bias)
    want = layer(inp.x).clone()
    layer.check_device_error()
    words = layer.fp8_ws[:4096].view(torch.int32)
    words[64:128] = 1  # counters of cut tiles
    words[0] = code
    layer.ws[:4].view(torch.int32)[0] = layer_code
    with pytest.raises(M.MoEError) as e:
        layer.check_device_error()
    assert e.value.status == (5 if layer_code else 6)
    assert not words.any()
    assert torch.equal(layer(inp.x), want)
    layer.check_device_error()


@pytest.mark.parametrize("kind", ["fp8", "bf16"])
def test_router_weight_changed_under_a_captured_forward(kind):
    """The graph routes by the router weight as resplit_router last split it, other tensors having
    come and gone in between."""
    shape = W.reduced(W.DSV3_DECODE, 64, 256, 128)
    inp = W.make_inputs(shape, device="cuda")
    cfg = M.config_from_shape(shape)
    assert M.router_split_size(cfg) > 0

    def layer_of(w_router):
        if kind == "bf16":
            return M.MoELayer(cfg, w_router, inp.w_gate, inp.w_up, inp.w_down, inp.logit_bias)
        return M.MoELayerFp8(cfg, w_router, M.Fp8Experts.quantize(inp.w_gate, inp.w_up, inp.w_down),
                             inp.logit_bias)

    w_router = inp.w_router.clone()
    layer = layer_of(w_router)
    graph = layer.capture(inp.x)
    graph.replay()
    before = layer.bufs.out.clone()
    w_router.copy_(inp.w_router.flip(1))
    layer.resplit_router()
    size = M.router_split_size(cfg)
    junk = [torch.full((size,), 0x5A, dtype=torch.uint8, device="cuda") for _ in range(4)]
    graph.replay()
    got = layer.bufs.out.clone()
    assert torch.equal(got, layer_of(w_router)(inp.x)) and not torch.equal(got, before)
    del junk


def test_grouped_gemm_of_the_most_rows():
    """2^31 - 128 rows, the most that are taken: whole tiles up to the last row."""
    rows, K, N = 2 ** 31 - 128, 16, 8
    if torch.cuda.mem_get_info()[0] < 100 * 2 ** 30:
        pytest.skip("needs 100 GB of free device memory")
    g = gen(9)
    a_q = torch.zeros((rows, K), dtype=torch.uint8, device="cuda").view(E4M3)
    a_s = torch.zeros((rows, 1), device="cuda")
    last_q, last_s = quantized_rows(torch.randn((300, K), generator=g))
    a_q.view(torch.uint8)[-300:] = last_q.view(torch.uint8)
    a_s[-300:] = last_s
    w_q, w_s = quantized_weights(torch.randn((1, N, K), generator=g))
    out = torch.full((rows, N), 3.25, dtype=torch.bfloat16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    ws = M.alloc_fp8_workspace()
    M.moe_fp8_grouped_gemm(a_q, a_s, torch.zeros(1, **i32), torch.full((1,), rows, **i32), w_q, w_s,
                           out, ws)
    M.moe_check_device_error(ws)
    check_product(out[-300:], last_q, last_s, w_q, w_s, [0], [300])
    for at in (0, 2 ** 30, 2 ** 31 - 1000):
        assert not out[at:at + 500].any()
    del a_q, a_s, out
    torch.cuda.empty_cache()


@pytest.mark.parametrize("slack", [0, 200], ids=["few-rows kernel", "many-rows kernel"])
@pytest.mark.parametrize("counts", [[32] * 8, [33, 0, 1, 64, 2, 0, 100, 56], [64, 0, 0, 64],
                                    [48, 0], [0, 0, 0, 65, 0, 0, 0, 63]])
def test_the_same_buckets_in_either_kernel(counts, slack):
    """The length of the buffers chooses the kernel; the buckets are the same.  What lies behind
    them, NaN here, has no part in the results."""
    N, K, E = 520, 1040, len(counts)
    first, used = starts(counts)
    rows = used if slack == 0 else 32 * E + slack
    a_q, a_s = quantized_rows(torch.randn((rows, K), generator=gen(3)).bfloat16())
    a_q.view(torch.uint8)[used:] = 0x7F
    a_s[used:] = float("nan")
    w_q, w_s = quantized_weights(torch.randn((E, N, K), generator=gen(4)) / K ** 0.5)
    out = torch.full((rows, N), 3.25, dtype=torch.bfloat16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    ws = M.alloc_fp8_workspace()
    M.moe_fp8_grouped_gemm(a_q, a_s, torch.tensor(first, **i32), torch.tensor(counts, **i32), w_q,
                           w_s, out, ws)
    M.moe_check_device_error(ws)
    check_product(out, a_q, a_s, w_q, w_s, first, counts)


@pytest.mark.parametrize("rows", [5, 40], ids=["few", "many"])
def test_scale_products_below_the_smallest_normal_number(rows):
    """a_scale w_scale is rounded to a multiple of 2^-149 there, off by at most 2^-150; a block's
    sum is at most 128 x 448^2 < 2^24.7, so a block adds at most 2^-125 to the error."""
    N, K = 136, 400
    g = gen(8)
    a = torch.randint(0, 256, (rows, K), generator=g, dtype=torch.uint8)
    w = torch.randint(0, 256, (1, N, K), generator=g, dtype=torch.uint8)
    for t in (a, w):
        t[(t & 0x7F) == 0x7F] = 0x7E  # (no NaN)
    a, w = a.cuda().view(E4M3), w.cuda().view(E4M3)
    a_s = torch.exp2(-80 - 20 * torch.rand((rows, 4), generator=g)).cuda()
    w_s = torch.exp2(-55 - 10 * torch.rand((1, 2, 4), generator=g)).cuda()
    out = torch.full((rows, N), 3.25, dtype=torch.bfloat16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    M.moe_fp8_grouped_gemm(a, a_s, torch.zeros(1, **i32), torch.full((1,), rows, **i32), w, w_s,
                           out, M.alloc_fp8_workspace())
    ref, mag = O.product(O.rows_value(a, a_s), O.weight_value(w[0], w_s[0]))
    assert (ref.abs() < 2.0 ** -105).all() and (ref.abs() > 2.0 ** -126).any()
    # bf16 rounds to multiples of 2^-133 below its smallest normal number
    room = (1 + O.BF16_HALF_STEP) * (O.sum_error(K) * mag + 4 * 2.0 ** -125)
    room = room + torch.clamp(O.BF16_HALF_STEP * ref.abs(), min=2.0 ** -134)
    assert ((out.cpu().double() - ref).abs() <= room).all()


@pytest.mark.parametrize("times", [1, 3], ids=["few", "many"])
def test_silu_of_far_gates(times):
    """Gates from -1000 to 1000, one to a row, times an up of 1: below -87.3 silu is 0, off by less
    than 2^-119."""
    gates = [-1000.0, -448.0, -104.0, -96.0, -90.0, -88.0, -87.5, -87.0, -80.0, -20.0, -1.0, -2e-3,
             0.0, 2e-3, 1.0, 20.0, 88.0, 100.0, 1000.0] * times
    R, d, f = len(gates), 256, 16
    x = torch.zeros((R, d))
    x[:, 0] = torch.tensor(gates)
    x[:, 128] = 1.0
    wg, wu = torch.zeros((1, f, d)), torch.zeros((1, f, d))
    wg[:, :, 0], wu[:, :, 128] = 1.0, 1.0
    x_q, x_s = quantized_rows(x)
    experts = M.Fp8Experts.quantize(wg.cuda(), wu.cuda(), torch.ones((1, d, f), device="cuda"))
    cfg = M.make_config(R, d, f, 1, 1)
    i32 = dict(dtype=torch.int32, device="cuda")
    h_q, h_s = torch.empty((R, f), device="cuda").to(E4M3), torch.empty((R, 1), device="cuda")
    y = torch.empty((R, d), dtype=torch.bfloat16, device="cuda")
    M.moe_expert_ffn_fp8(cfg, x_q, x_s, torch.tensor([0, R], **i32), torch.full((1,), R, **i32),
                         experts, h_q, h_s, y, M.alloc_fp8_workspace())
    v = O.rows_value(x_q, x_s)
    g = O.product(v, O.weight_value(experts.w_gate[0], experts.gate_scale[0]))[0]
    u = O.product(v, O.weight_value(experts.w_up[0], experts.up_scale[0]))[0]
    ref = g * torch.sigmoid(g) * u
    # Gate and up have one product each: two roundings of 2^-24, and silu moves by at most 1 + |g|
    # of itself for as much of g.  The fast exp of -g is off by up to 2 + 1.2 |g| units of 2^-23.  32
    # steps for the division and the products, as in test_ffn.
    room = (2 * (1 + g.abs()) + 2 + 2 * (2 + 1.2 * g.abs()) + 32) * 2.0 ** -24 * ref.abs()
    room = room + 2.0 ** -119 * u.abs()
    # the entries of a row are alike: its scale is |h| / 448, or that of 2^-100
    step = torch.maximum(O.E4M3_HALF_STEP * ref.abs(), torch.tensor(2.0 ** -110 / 448).double())
    step[ref.abs() > 2.0 ** -99] = 0.0  # q = 448: the largest entry maps to itself
    off = (O.rows_value(h_q, h_s) - ref).abs()
    assert (off <= room + (1 + 2.0 ** -15) * step).all(), (off / (room + step)).max()
    assert (O.rows_value(h_q, h_s)[:3] == 0).all()
