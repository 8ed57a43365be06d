"""MXFP4: quantisation and its values (bit for bit), and the product of two such matrices.

The product is compared with the sum in 64 bits of the values the codes stand
for. Tolerance: every product of two codes and scales is exact; a tensor-core
step adds 64 of them to the running sum, which may drop up to one step (2^-23)
of the largest magnitude it meets, at most S = sum |x w|, per block of 32; then
the output's rounding (2^-8 for bf16, 2^-24 for fp32):
(D / 32 + 1) 2^-23 S + h |y|.
"""
import ctypes
import math

import pytest
import torch

import vocab_wide_logprobs_gb300 as vp
from vocab_wide_logprobs_gb300 import _lib

OK, ERR_NULL, ERR_SHAPE, ERR_DTYPE, ERR_LAYOUT, ERR_ALIGN, ERR_LAUNCH, ERR_ARG, ERR_DEVICE = range(9)
MAGNITUDES = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def plain_quantize(x):
    """(codes [N, D] 0..15, scale bytes [N, D / 32]) from the definition, in 64 bits."""
    N, D = x.shape
    b = x.double().reshape(N, D // 32, 32)
    amax = b.abs().amax(-1)
    bad = ~torch.isfinite(amax)
    e = torch.frexp(torch.where(bad, 1.0, amax))[1].double() - 3                # floor(log2 amax) - 2
    e = torch.where(amax == 0, -127.0, e).clamp(-127, 127)
    v = (b / torch.exp2(e)[..., None]).abs()
    dist = (v[..., None] - MAGNITUDES).abs()
    near = dist == dist.amin(-1, keepdim=True)
    # of two equally near magnitudes the one with an even index
    rank = torch.where(near, torch.arange(8) % 2, 9)
    code = rank.argmin(-1)
    code = torch.where(bad[..., None], 0, code + 8 * torch.signbit(b).long())
    return code.reshape(N, D), torch.where(bad, 255, (e + 127).long())


def plain_values(code, byte):
    v = MAGNITUDES[code % 8] * torch.where(code >= 8, -1.0, 1.0)
    s = torch.where(byte == 255, math.nan, torch.exp2(byte.double() - 127))
    return (v.reshape(code.shape[0], -1, 32) * s[..., None]).reshape(code.shape)


def pack(code, byte):
    """The public layout, placed byte by byte."""
    N, D = code.shape
    codes = (code[:, 0::2] + 16 * code[:, 1::2]).to(torch.uint8)
    scales = torch.zeros(-(-N // 128) * -(-D // 128) * 512, dtype=torch.uint8)
    r, b = torch.arange(N)[:, None], torch.arange(D // 32)[None, :]
    at = (r // 128 * -(-D // 128) + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4
    scales[at.reshape(-1)] = byte.reshape(-1).to(torch.uint8)
    return codes, scales


def inputs(N, D, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(N, D, generator=g) * torch.exp2(torch.randint(-6, 7, (N, D // 32), generator=g).float()
                                                    ).repeat_interleave(32, 1)
    special = [0.0, -0.0, 2.0 ** -126, 2.0 ** -130, 3.0e38, -3.0e38]
    for i, v in enumerate(special):
        row, block = i % N, i % (D // 32)
        x[row, 32 * block:32 * block + 32] = v
    if N > 6:                                                                   # ties and borders against a maximum of 4
        ties = torch.tensor([4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 7.9, 0.2499, 0.2501, 6.0, 6.5, 3.49, 3.51])
        x[6, :32] = torch.cat((ties, -ties))
        x[6, 32:64] = torch.cat((ties, -ties)).clamp(-4, 4)
    if N > 8:
        x[7, 5], x[8, 40] = math.nan, -math.inf
    return x.to(dtype)


SHAPES = [(1, 64), (3, 2112), (9, 128), (130, 192), (257, 64), (128, 320), (31, 4096)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", SHAPES)
def test_quantize_bit_for_bit(shape, dtype):
    N, D = shape
    x = inputs(N, D, dtype, N + D)
    code, byte = plain_quantize(x)
    ref_codes, ref_scales = pack(code, byte)
    wide = torch.zeros(N, D + 3, dtype=dtype, device="cuda")                    # rows at odd offsets
    wide[:, 1:D + 1] = x.cuda()
    for xg in (x.cuda(), wide[:, 1:D + 1]):
        codes, scales = vp.vp_mxfp4_quantize(xg)
        assert torch.equal(codes.cpu(), ref_codes) and torch.equal(scales.cpu(), ref_scales)
    for out in (torch.float32, torch.bfloat16):
        v = vp.vp_mxfp4_dequantize(codes, scales, dtype=out).cpu()
        ref = plain_values(code, byte)
        assert torch.equal(torch.nan_to_num(v.double(), 7.0), torch.nan_to_num(ref, 7.0))
        assert torch.equal(torch.isnan(v), torch.isnan(ref))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantize_does_not_depend_on_where_rows_begin(dtype):
    N, D = 13, 1088
    x = inputs(N, D, dtype, 77).cuda()
    ref = vp.vp_mxfp4_quantize(x)
    for offset in (1, 4, 8, 16):
        for gap in (0, 4, 8, 13, 16):
            room = torch.full((offset + N * (D + gap),), math.nan, dtype=dtype, device="cuda")
            view = room[offset:].view(N, D + gap)[:, :D]
            view.copy_(x)
            assert all(torch.equal(a, b) for a, b in zip(vp.vp_mxfp4_quantize(view), ref)), (offset, gap)


@pytest.mark.gpu
def test_quantize_rows_of_a_batch():
    """[B, T, D] rows with two strides, and caller's buffers."""
    x = torch.randn(3, 6, 128).to(torch.bfloat16).cuda()
    codes = torch.full((15, 64), 99, dtype=torch.uint8, device="cuda")
    scales = torch.full((512,), 99, dtype=torch.uint8, device="cuda")
    got = vp.vp_mxfp4_quantize(x[:, :-1], codes=codes, scales=scales)
    ref = vp.vp_mxfp4_quantize(x[:, :-1].reshape(15, 128))
    assert got[0].data_ptr() == codes.data_ptr() and all(torch.equal(a, b) for a, b in zip(got, ref))


def product_case(N, V, D, seed, spread=3):
    g = torch.Generator().manual_seed(seed)
    mats = []
    for rows in (N, V):
        code = torch.randint(0, 16, (rows, D), generator=g)
        byte = torch.randint(127 - spread, 128 + spread, (rows, D // 32), generator=g)
        mats.append((code, byte))
    return mats


def check_product(y, mats, dtype):
    x, w = (plain_values(*m) for m in mats)
    ref, size = x @ w.t(), x.abs() @ w.abs().t()
    tol = (x.shape[1] / 32 + 1) * 2.0 ** -23 * size + torch.finfo(dtype).eps / 2 * ref.abs()
    assert y.dtype == dtype and y.shape == ref.shape
    off = (y.double().cpu() - ref).abs() - tol
    assert off.max() <= 0, f"{float(off.max())} over its tolerance"


def gpu(mats):
    return [t.cuda() for m in mats for t in pack(*m)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(1, 1, 64), (1, 128, 128), (2, 5, 192), (16, 129, 256), (17, 1000, 320), (33, 127, 64),
                                   (64, 300, 1088), (65, 5003, 512), (128, 256, 256), (129, 255, 320), (300, 700, 2112),
                                   (1, 40000, 640), (520, 1300, 384)])
def test_product_against_64_bits(shape, dtype):
    mats = product_case(*shape, seed=sum(shape))
    check_product(vp.vp_linear_mxfp4_fwd(*gpu(mats), dtype=dtype), mats, dtype)
    assert vp.vp_fault_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(513, 20001, 320), (700, 13001, 832), (20, 60001, 192), (50, 60001, 576), (100, 60001, 192)])
def test_several_tiles_for_each_pair_and_cta(shape, dtype):
    """More tiles than run at once, two or three times over: both accumulators, their shared columns and the ring go round."""
    mats = product_case(*shape, seed=sum(shape))
    bufs = gpu(mats)
    y = vp.vp_linear_mxfp4_fwd(*bufs, dtype=dtype)
    check_product(y, mats, dtype)
    assert torch.equal(vp.vp_linear_mxfp4_fwd(*bufs, dtype=dtype).view(torch.int16), y.view(torch.int16))
    assert vp.vp_fault_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("N", [1, 20, 200, 513])
def test_product_of_quantised_matrices(N):
    g = torch.Generator().manual_seed(N)
    h, w = torch.randn(N, 448, generator=g).to(torch.bfloat16), (torch.randn(650, 448, generator=g) * 0.02)
    y = vp.vp_linear_mxfp4_fwd(*vp.vp_mxfp4_quantize(h.cuda()), *vp.vp_mxfp4_quantize(w.cuda()), dtype=torch.float32)
    check_product(y, [plain_quantize(h), plain_quantize(w)], torch.float32)


@pytest.mark.gpu
@pytest.mark.parametrize("N", [3, 70, 300])
def test_each_code_and_block_lands_where_it_belongs(N):
    """One element each in x and w: a product of exactly one pair, for every place in a stage and in the scale tiles."""
    D, V = 512, 260
    code_x, code_w = torch.zeros(N, D, dtype=torch.int64), torch.zeros(V, D, dtype=torch.int64)
    byte_x, byte_w = torch.full((N, D // 32), 127), torch.full((V, D // 32), 127)
    for n in range(N):
        code_x[n, (37 * n + 5) % D] = 1 + n % 7
        byte_x[n] = 120 + (torch.arange(D // 32) + n) % 13
    for v in range(V):
        code_w[v] = (torch.arange(D) + v) % 16
        byte_w[v] = 119 + (3 * torch.arange(D // 32) + v) % 17
    mats = [(code_x, byte_x), (code_w, byte_w)]
    y = vp.vp_linear_mxfp4_fwd(*gpu(mats), dtype=torch.float32)
    assert torch.equal(y.double().cpu(), plain_values(*mats[0]) @ plain_values(*mats[1]).t())


@pytest.mark.gpu
@pytest.mark.parametrize("N", [2, 40, 300])
def test_a_nan_scale_stays_in_its_row(N):
    mats = product_case(N, 300, 256, seed=N)
    mats[0][1][1, 3] = 255
    mats[1][1][270, 0] = 255
    y = torch.isnan(vp.vp_linear_mxfp4_fwd(*gpu(mats), dtype=torch.float32)).cpu()
    ref = torch.zeros(N, 300, dtype=torch.bool)
    ref[1], ref[:, 270] = True, True
    assert torch.equal(y, ref)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_an_element_does_not_depend_on_the_batch(dtype):
    N, V, D = 700, 1000, 1344
    mats = product_case(N, V, D, seed=4, spread=9)
    whole = vp.vp_linear_mxfp4_fwd(*gpu(mats), dtype=dtype)
    for n in (1, 16, 31, 64, 100, 129, 256, 300):
        first = [(mats[0][0][:n], mats[0][1][:n]), mats[1]]
        part = vp.vp_linear_mxfp4_fwd(*gpu(first), dtype=dtype)
        assert torch.equal(part.view(torch.int16), whole[:n].view(torch.int16)), n


@pytest.mark.gpu
def test_streams_and_graphs():
    mats = product_case(40, 900, 512, seed=1)
    bufs = gpu(mats)
    ref = vp.vp_linear_mxfp4_fwd(*bufs)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = vp.vp_linear_mxfp4_fwd(*bufs)
    side.synchronize()
    assert torch.equal(got, ref)
    h = torch.randn(40, 512, device="cuda").to(torch.bfloat16)
    want = vp.vp_linear_mxfp4_fwd(*vp.vp_mxfp4_quantize(h), *bufs[2:])
    held = torch.zeros_like(h)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = vp.vp_linear_mxfp4_fwd(*vp.vp_mxfp4_quantize(held), *bufs[2:])
    held.copy_(h)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and vp.vp_fault_status() == 0


@pytest.mark.gpu
@pytest.mark.slow
@pytest.mark.parametrize("shape", [(1, 2 ** 31 - 100), (2 ** 31 - 100, 1)])
def test_as_many_rows_as_the_calls_take(shape):
    """Row counts that a tile's worth more would carry past 31 bits, of W for single CTAs and of x for the pairs."""
    N, V = shape
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GB")
    few = product_case(1, 1, 64, seed=1)
    long, short = torch.zeros(2 ** 31 - 100, 32, dtype=torch.uint8, device="cuda"), gpu(few)[:2]
    scales = torch.full((vp.vp_mxfp4_scale_bytes(2 ** 31 - 100, 64),), 127, dtype=torch.uint8, device="cuda")
    at = torch.tensor([0, 127, 128, 2 ** 30 + 3, 2 ** 31 - 356, 2 ** 31 - 129, 2 ** 31 - 101], device="cuda")
    long[at] = torch.randint(0, 256, (at.numel(), 32), dtype=torch.uint8, device="cuda")
    y = torch.full((N, V), math.nan, dtype=torch.bfloat16, device="cuda")
    big = (long, scales)
    args = (*short, *big) if N == 1 else (*big, *short)
    vp.vp_linear_mxfp4_fwd(*args, y=y)
    y = y.view(-1)
    codes = torch.stack((long[at] % 16, long[at] // 16), 2).view(-1, 64).cpu().long()
    values = plain_values(codes, torch.full((at.numel(), 2), 127)) @ plain_values(*few[0])[0]
    assert (y[at].cpu().double() - values).abs().max() <= 2.0 ** -8 * values.abs().max() + 3 * 2.0 ** -23 * 36 * 64 * 8
    y[at] = 0
    assert not y.any()
    assert vp.vp_fault_status() == 0


# ---------------------------------------------------------------------------
# refusals (CPU)
# ---------------------------------------------------------------------------
FAKE, FAKE_ODD = ctypes.c_void_p(0x100000), ctypes.c_void_p(0x100001)      # never dereferenced
FAKE_8 = ctypes.c_void_p(0x100008)


def test_entry_points_check_arguments_on_the_host():
    L = _lib.lib()

    def quant(x=FAKE, dtype=1, N=4, D=64, s_i=64, codes=FAKE, scales=FAKE):
        return L.vp_mxfp4_quantize(x, dtype, N, D, 4, 0, s_i, codes, scales, None)

    assert quant(dtype=3) == ERR_DTYPE
    assert quant(D=32) == ERR_SHAPE and quant(D=96) == ERR_SHAPE and quant(D=1 << 21) == ERR_SHAPE
    assert quant(N=-1) == ERR_SHAPE and quant(s_i=-64) == ERR_LAYOUT
    assert quant(x=None) == ERR_NULL and quant(codes=None) == ERR_NULL and quant(scales=None) == ERR_NULL
    assert quant(x=FAKE_ODD) == ERR_ALIGN and quant(codes=FAKE_8) == ERR_ALIGN and quant(scales=FAKE_8) == ERR_ALIGN
    assert quant(N=0, x=None, codes=None, scales=None) == OK
    assert L.vp_mxfp4_dequantize(FAKE, FAKE, 4, 64, 5, FAKE, None) == ERR_DTYPE
    assert L.vp_mxfp4_dequantize(FAKE, FAKE, 4, 65, 1, FAKE, None) == ERR_SHAPE
    assert L.vp_mxfp4_dequantize(FAKE, None, 4, 64, 1, FAKE, None) == ERR_NULL
    assert L.vp_mxfp4_dequantize(FAKE, FAKE, 4, 64, 1, FAKE_8, None) == ERR_ALIGN
    four = (FAKE, FAKE, FAKE, FAKE)
    assert L.vp_linear_mxfp4_fwd(*four, 4, 16, 64, 2, FAKE, None) == ERR_DTYPE
    assert L.vp_linear_mxfp4_fwd(*four, 4, 0, 64, 0, FAKE, None) == ERR_SHAPE
    assert L.vp_linear_mxfp4_fwd(*four, 4, 16, 100, 0, FAKE, None) == ERR_SHAPE
    assert L.vp_linear_mxfp4_fwd(FAKE, FAKE, FAKE, None, 4, 16, 64, 0, FAKE, None) == ERR_NULL
    assert L.vp_linear_mxfp4_fwd(FAKE, FAKE, FAKE_8, FAKE, 4, 16, 64, 0, FAKE, None) == ERR_ALIGN
    assert L.vp_linear_mxfp4_fwd(*four, 4, 16, 64, 1, FAKE_ODD, None) == ERR_ALIGN
    assert L.vp_linear_mxfp4_fwd(None, None, None, None, 0, 16, 64, 1, None, None) == OK
    assert vp.vp_mxfp4_scale_bytes(1, 64) == 512 and vp.vp_mxfp4_scale_bytes(129, 192) == 4 * 512
    assert vp.vp_mxfp4_scale_bytes(4, 96) == 0


def status(fn):
    with pytest.raises(vp.VPError) as e:
        fn()
    return e.value.status


def test_binding_checks_tensors():
    x = torch.zeros(4, 128)
    codes, scales = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8)
    assert status(lambda: vp.vp_mxfp4_quantize(torch.zeros(4, 96))) == ERR_SHAPE
    assert status(lambda: vp.vp_mxfp4_quantize(x, codes=codes[:3])) == ERR_SHAPE
    assert status(lambda: vp.vp_mxfp4_quantize(x, scales=scales[:511])) == ERR_SHAPE
    assert status(lambda: vp.vp_mxfp4_quantize(x.t())) in (ERR_SHAPE, ERR_LAYOUT)
    assert status(lambda: vp.vp_mxfp4_dequantize(codes, scales[:-1])) == ERR_SHAPE
    assert status(lambda: vp.vp_mxfp4_dequantize(codes.int(), scales)) == ERR_DTYPE
    assert status(lambda: vp.vp_mxfp4_dequantize(codes, scales, dtype=torch.float16)) == ERR_DTYPE
    assert status(lambda: vp.vp_mxfp4_dequantize(codes[:, :40].contiguous(), scales)) == ERR_SHAPE
    assert status(lambda: vp.vp_linear_mxfp4_fwd(codes, scales, codes[:, :32].contiguous(), scales)) == ERR_SHAPE
    assert status(lambda: vp.vp_linear_mxfp4_fwd(codes, scales, codes, scales, y=torch.zeros(4, 4))) == ERR_DTYPE
    for call in (lambda: vp.vp_mxfp4_quantize(x), lambda: vp.vp_mxfp4_dequantize(codes, scales),
                 lambda: vp.vp_linear_mxfp4_fwd(codes, scales, codes, scales)):
        assert status(call) == ERR_DEVICE


def test_plain_quantiser_by_hand():
    x = torch.zeros(1, 64)
    x[0, :8] = torch.tensor([6.0, 5.0, 3.5, 2.5, 1.75, 1.25, 0.75, -0.25])
    x[0, 32:36] = torch.tensor([7.9, -2.0 ** -3, 1.0, 0.24])
    code, byte = plain_quantize(x)
    assert code[0, :8].tolist() == [7, 6, 6, 4, 4, 2, 2, 8] and byte.tolist() == [[127, 127]]
    assert plain_values(code, byte)[0, 32:36].tolist() == [6.0, -0.0, 1.0, 0.0]
