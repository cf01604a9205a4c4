"""The product of few tokens with grouped 4-bit integer weights, against 64 bits."""
import itertools

import pytest
import torch

import precision_tensor_core_gb300 as ptc
from tests.gpu_util import DEV
from tests.s4_ref import check, gen, matrix, rand, weights

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(DEV)
    yield
    for k in ("s4_tokens_rows", "s4_tokens_split", "s4_tokens_tiles"):
        ptc.ptc_set_tuning(k, 0)
    assert ptc.gemm_poll_device_error() == ptc.PTC_OK


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("group", [32, 64, 128, 256])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M, N, K", [(1, 1, 1), (1, 17, 31), (2, 16, 128), (3, 100, 257), (8, 33, 1000), (9, 130, 640),
                                     (16, 300, 2090), (17, 40, 129), (50, 64, 384), (1, 4096, 512)])
def test_sizes(M, N, K, group, zeros, dtype):
    w = weights(M + N, (), N, K, group, zeros, dtype)
    x = rand(K, M, K, dtype=dtype)
    check(ptc.matmul_a16_s4(x, matrix(w)), x, w, dtype)


@pytest.mark.parametrize("xt, st", [(BF, HF), (HF, BF)])
def test_scales_of_the_other_type(xt, st):
    w = weights(1, (), 200, 777, 64, True, st)
    x = rand(2, 5, 777, dtype=xt)
    check(ptc.matmul_a16_s4(x, matrix(w)), x, w, xt)


SHAPES = list(itertools.product([1, 2, 4, 8, 16], [1, 2, 4, 8], [1, 2]))


@pytest.mark.parametrize("rows, split, tiles", SHAPES)
@pytest.mark.parametrize("group", [32, 128])
def test_every_launch_shape(rows, split, tiles, group):
    """K of 128 stages and a part: every share has its stages.  The shape is the one asked for where its
    activations fit, up to four tokens in all of them."""
    N, K = 200, 33000
    w = weights(3, (), N, K, group, True, HF)
    for M in (1, 4, 16):
        x = rand(4, M, K, dtype=HF)
        for k, v in (("rows", rows), ("split", split), ("tiles", tiles)):
            ptc.ptc_set_tuning("s4_tokens_" + k, v)
        got = ptc.matmul_a16_s4(x, matrix(w))
        grid, cluster, ks, tile = ptc.ptc_last_fp4_launch()
        if M <= 4:
            assert (cluster, ks, tile) == (split, split, 16 * rows * tiles) and grid == -(-N // tile) * split
        check(got, x, w, HF)
    for k in ("rows", "split", "tiles"):
        ptc.ptc_set_tuning("s4_tokens_" + k, 0)


@pytest.mark.parametrize("M, N, K", [(1, 4096, 4096), (16, 2048, 8192), (4, 512, 8192), (2, 64, 40000), (16, 24, 70000)])
def test_larger(M, N, K):
    w = weights(5, (), N, K, 128, False, BF)
    x = rand(6, M, K, dtype=BF)
    check(ptc.matmul_a16_s4(x, matrix(w)), x, w, BF)


@pytest.mark.parametrize("rows, split, tiles", [(1, 1, 1), (1, 1, 2), (4, 2, 1), (8, 4, 2), (8, 1, 1)])
@pytest.mark.parametrize("M, K, group", [(1, 2100, 128), (3, 2048, 32), (16, 4096, 256), (40, 2100, 64)])
def test_many_row_tiles_per_cta(rows, split, tiles, M, K, group):
    """Every CTA walks over several tiles of rows, the last ones partial."""
    N = 30011
    w = weights(32, (), N, K, group, group == 32, BF)
    x = rand(33, M, K, dtype=BF)
    for k, v in (("rows", rows), ("split", split), ("tiles", tiles)):
        ptc.ptc_set_tuning("s4_tokens_" + k, v)
    got = ptc.matmul_a16_s4(x, matrix(w))
    for k in ("rows", "split", "tiles"):
        ptc.ptc_set_tuning("s4_tokens_" + k, 0)
    check(got, x, w, BF)


@pytest.mark.parametrize("M, N, K", [(3, 500, 2090), (16, 2000, 4096), (16, 64, 40000), (23, 300, 900)])
def test_without_workspace(M, N, K):
    """Every CTA making the operands itself gives the same bits."""
    w = weights(34, (), N, K, 64, True, HF)
    x, m = rand(35, M, K, dtype=HF), matrix(w)
    want = ptc.matmul_a16_s4(x, m)
    got = torch.empty_like(want)
    assert ptc.gemm_a16_s4_workspace(M, K) > 0 and ptc.gemm_a16_s4_workspace(2, K) == 0
    ptc.gemm_a16_s4(M, N, K, ptc.PTC_OUT_F16, x.data_ptr(), K, m.codes.data_ptr(), m.codes.stride(0), 64, ptc.PTC_OUT_F16,
                    m.scales.data_ptr(), m.zeros.data_ptr(), got.data_ptr(), N, stream=torch.cuda.current_stream().cuda_stream)
    assert torch.equal(got, want)


def test_codes_one_by_one():
    """Every code at every place of a block with activations that pick one place: exact."""
    codes = torch.arange(16, device=DEV, dtype=torch.uint8)
    K = 256
    c = ((codes | (codes << 4)).unsqueeze(1).expand(16, K // 2)).contiguous()
    scales = torch.ones(16, K // 128, device=DEV, dtype=HF)
    m = ptc.S4Matrix(c, ptc.S4Matrix.tile_scales(scales), K)
    signed = torch.where(codes > 7, codes.int() - 16, codes.int()).double()
    for first in range(0, K, 16):
        x = torch.zeros(16, K, device=DEV, dtype=HF)
        x[torch.arange(16), first + torch.arange(16)] = 1.5
        assert torch.equal(ptc.matmul_a16_s4(x, m).double(), (1.5 * signed).expand(16, 16))


@pytest.mark.parametrize("dtype", [BF, HF])
def test_range_of_activations(dtype):
    """Each token at its own size, from the type's smallest to its largest numbers, and blocks of very different sizes."""
    lo, hi = (-120, 118) if dtype == BF else (-14, 8)
    K = 512
    w = weights(7, (), 96, K, 32, False, dtype)
    e = torch.linspace(lo, hi, 16, device=DEV).round()
    x = (rand(8, 16, K).clamp(-4, 4).double() * torch.exp2(e.double()).unsqueeze(1)).to(dtype)
    got = ptc.matmul_a16_s4(x, matrix(w))
    want = x.double() @ w["values"].t()
    fits = want.abs() < torch.finfo(dtype).max
    size = x.double().abs() @ w["size"].t()
    least = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    bound = torch.finfo(dtype).eps / 2 * want.abs() + 2.0 ** -17 * size + least
    assert bool(((got.double() - want).abs() <= bound)[fits].all())
    # one element far above the rest of its block: the others count down to 2^-28 of it
    x = rand(9, 2, K, dtype=dtype)
    x[:, 40] = 2.0 ** 10
    check(ptc.matmul_a16_s4(x, matrix(w)), x, w, dtype)


def test_small_and_zero_blocks():
    w = weights(10, (), 50, 320, 64, True, BF)
    x = rand(11, 6, 320, dtype=BF)
    x[0] = 0
    x[1, 64:128] = 0
    x[2] = 0
    x[2, 77] = 2.0 ** -133  # bfloat16's smallest
    x[3, :300] = 0
    got = ptc.matmul_a16_s4(x, matrix(w))
    assert not got[0].any()
    check(got, x, w, BF)


def test_not_finite():
    """A token with an infinity or NaN is NaN; no other token changes; a scale's NaN stays in its row."""
    w = weights(12, (), 60, 500, 32, False, HF)
    x = rand(13, 12, 500, dtype=HF)
    clean = ptc.matmul_a16_s4(x, matrix(w))
    x[3, 17], x[9, 499] = float("inf"), float("nan")
    got = ptc.matmul_a16_s4(x, matrix(w))
    keep = [i for i in range(12) if i not in (3, 9)]
    assert torch.equal(got[keep], clean[keep]) and bool(got[[3, 9]].isnan().all())
    w["scales"][7, 2] = float("nan")
    got = ptc.matmul_a16_s4(x, matrix(w))
    rows = [i for i in range(60) if i != 7]
    assert torch.equal(got[keep][:, rows], clean[keep][:, rows]) and bool(got[:, 7].isnan().all())


def test_views_and_out():
    """Activations, codes and results as column slices, rows that are not aligned; what lies beside the result stays."""
    w = weights(14, (), 77, 300, 128, True, BF, slack=3)
    buf = rand(15, 9, 1001, dtype=BF)
    for at in (0, 8, 13):
        x = buf[:, at:at + 300]
        b = torch.full((9, 200), 7.0, device=DEV, dtype=BF)
        out = b[:, 61:138]
        got = ptc.matmul_a16_s4(x, matrix(w), out=out)
        assert got is out
        check(got, x, w, BF)
        assert bool((b[:, :61] == 7).all()) and bool((b[:, 138:] == 7).all())
    wide = torch.zeros(77, 4096, device=DEV, dtype=torch.uint8)
    wide[:, 160:320] = w["codes"][:, :160]
    m = ptc.S4Matrix(wide[:, 160:310], ptc.S4Matrix.tile_scales(w["scales"]), 300, 128, ptc.S4Matrix.tile_scales(w["zeros"]))
    check(ptc.matmul_a16_s4(buf[:, 5:305], m), buf[:, 5:305], w, BF)


def test_nothing_past_the_rows_is_used():
    """Nibbles past K, and tiles' entries past the rows, may hold anything, NaN among it."""
    w = weights(16, (), 21, 333, 32, True, HF)
    x = rand(17, 4, 333, dtype=HF)
    s, z = (ptc.S4Matrix.tile_scales(w[k]).view(2, -1, 16) for k in ("scales", "zeros"))
    s[1, :, 5:] = float("nan")
    z[1, :, 5:] = float("inf")
    got = ptc.matmul_a16_s4(x, ptc.S4Matrix(w["codes"], s.view(-1), 333, 32, z.view(-1)))
    check(got, x, w, HF)


def test_empty():
    m = matrix(weights(18, (), 40, 128, 128))
    assert ptc.matmul_a16_s4(torch.empty(0, 128, device=DEV, dtype=BF), m).shape == (0, 40)
    none = ptc.S4Matrix(torch.empty(40, 0, device=DEV, dtype=torch.uint8), torch.empty(0, device=DEV, dtype=BF), 0)
    assert not ptc.matmul_a16_s4(torch.empty(3, 0, device=DEV, dtype=BF), none).any()
    no_rows = ptc.S4Matrix(torch.empty(0, 64, device=DEV, dtype=torch.uint8), torch.empty(0, device=DEV, dtype=BF), 128)
    assert ptc.matmul_a16_s4(torch.ones(3, 128, device=DEV, dtype=BF), no_rows).shape == (3, 0)


def test_quantize():
    """Weights rounded when they are loaded: within half a step of a group's scale, and exact for codes times scales."""
    for zeros, group in ((False, 32), (True, 128), (False, 512)):
        w = rand(19, 3, 40, 500)
        m = ptc.S4Matrix.quantize(w, group, zeros)
        assert m.shape == (3, 40, 500) and m.group == group and (m.zeros is not None) == zeros
        for e in range(3):
            one = ptc.S4Matrix(m.codes[e], m.scales.view(3, -1)[e], 500, group, None if m.zeros is None else m.zeros.view(3, -1)[e])
            eye = torch.eye(500, device=DEV, dtype=BF)
            back = ptc.matmul_a16_s4(eye, one).t().float()
            step = torch.nn.functional.pad(w[e], (0, -500 % group)).view(40, -1, group)
            step = (step.amax(-1).clamp(min=0) - step.amin(-1).clamp(max=0)) / 15 if zeros else step.abs().amax(-1) / 7
            # half a step (a whole one where a rounded zero or scale clips the ends), the scale's and the result's rounding
            bound = step.repeat_interleave(group, 1)[:, :500] * (1.0 if zeros else 0.5) + w[e].abs() * 2.0 ** -6
            assert bool(((back - w[e]).abs() <= bound).all())
    assert not ptc.matmul_a16_s4(torch.ones(2, 64, device=DEV, dtype=BF), ptc.S4Matrix.quantize(torch.zeros(5, 64, device=DEV), 32, True)).any()


def test_graph_and_streams():
    w = weights(20, (), 400, 3000, 128, False, BF)
    m, x = matrix(w), rand(21, 4, 3000, dtype=BF)
    want = ptc.matmul_a16_s4(x, m)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = ptc.matmul_a16_s4(x, m, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ptc.matmul_a16_s4(x, m)
    keep = x.clone()
    x.zero_()
    graph.replay()
    assert not got.any()
    x.copy_(keep)
    graph.replay()
    assert torch.equal(got, want)


def test_codes_past_32_bit_offsets():
    """Rows whose offsets exceed 2^32 bytes, by their pitch."""
    w = weights(22, (), 40, 200, 64, False, BF)
    pitch = 120 * (1 << 20)
    buf = torch.empty(40 * pitch, dtype=torch.uint8, device=DEV)
    v = buf.as_strided((40, 112), (pitch, 1))
    v.copy_(w["codes"])
    x = rand(23, 3, 200, dtype=BF)
    got = ptc.matmul_a16_s4(x, ptc.S4Matrix(v, ptc.S4Matrix.tile_scales(w["scales"]), 200, 64))
    check(got, x, w, BF)


def test_weights_that_never_arrive_are_reported():
    """A wait that runs out ends the call and is reported; the next call is whole."""
    w = weights(30, (), 300, 4000, 128, False, BF)
    m, x = matrix(w), rand(31, 3, 4000, dtype=BF)
    for split in (1, 2):
        ptc.ptc_set_tuning("s4_tokens_split", split)
        want = ptc.matmul_a16_s4(x, m)
        torch.cuda.synchronize()
        ptc.ptc_debug_set_wait_limit(20_000_000, 1)
        try:
            ptc.matmul_a16_s4(x, m)
            torch.cuda.synchronize()
            assert ptc.lib().gemm_poll_device_error() == ptc.PTC_ERR_TIMEOUT
        finally:
            ptc.ptc_debug_set_wait_limit(0, -1)
            ptc.ptc_set_tuning("s4_tokens_split", 0)
        ptc.ptc_set_tuning("s4_tokens_split", split)
        assert torch.equal(ptc.matmul_a16_s4(x, m), want)
        ptc.ptc_set_tuning("s4_tokens_split", 0)


def test_refusals():
    w = weights(24, (), 32, 256, 128, True, BF)
    s, z = ptc.S4Matrix.tile_scales(w["scales"]), ptc.S4Matrix.tile_scales(w["zeros"])
    c, m = w["codes"], matrix(w)
    x = rand(25, 2, 256, dtype=BF)
    many = ptc.S4Matrix(c.unsqueeze(0), s, 256)
    bad = [
        (TypeError, lambda: ptc.S4Matrix(c.char(), s, 256)), (TypeError, lambda: ptc.S4Matrix(c, s.float(), 256)),
        (ValueError, lambda: ptc.S4Matrix(c, s, 257)), (ValueError, lambda: ptc.S4Matrix(c, s, 256, 48)),
        (ValueError, lambda: ptc.S4Matrix(c, s, 256, 0)), (ValueError, lambda: ptc.S4Matrix(c, s, 256, 192)),
        (ValueError, lambda: ptc.S4Matrix(c, s[:-16], 256)), (ValueError, lambda: ptc.S4Matrix(c, s, 256, 128, z[:-16])),
        (ValueError, lambda: ptc.S4Matrix(c, s, 256, 128, z.half())), (ValueError, lambda: ptc.S4Matrix(c[:, ::2], s, 128)),
        (ValueError, lambda: ptc.S4Matrix(torch.empty(32, 136, device=DEV, dtype=torch.uint8), s, 256)),
        (ValueError, lambda: ptc.S4Matrix(c.cpu(), s, 256)), (ValueError, lambda: ptc.S4Matrix(c, s.cpu(), 256)),
        (ValueError, lambda: ptc.S4Matrix(c[0], s, 256)), (ValueError, lambda: ptc.S4Matrix(c, s, -1)),
        (TypeError, lambda: ptc.matmul_a16_s4(x.float(), m)), (ValueError, lambda: ptc.matmul_a16_s4(x[:, :255], m)),
        (TypeError, lambda: ptc.matmul_a16_s4(x, c)), (ValueError, lambda: ptc.matmul_a16_s4(x, many)),
        (ValueError, lambda: ptc.matmul_a16_s4(x.cpu(), m)), (ValueError, lambda: ptc.matmul_a16_s4(x, m, out=x.half()[:, :32])),
        (ValueError, lambda: ptc.matmul_a16_s4(x, m, out=x[:, :31])), (ptc.PtcError, lambda: ptc.matmul_a16_s4(x, m, out=x[:, :32])),
        (RuntimeError, lambda: ptc.matmul_a16_s4(rand(1, 2, 256).to(BF).requires_grad_(), m)),
        (ptc.PtcError, lambda: ptc.matmul_a16_s4(x, ptc.S4Matrix(torch.zeros(1 << 13, device=DEV, dtype=torch.uint8)[8:8 + 4096].view(32, 128), s, 256))),
    ]
    for i, (error, call) in enumerate(bad):
        with pytest.raises(error):
            call()
            print("not refused:", i)


@pytest.mark.parametrize("seed", range(12))
def test_random_sizes(seed):
    g = torch.Generator().manual_seed(seed)
    M, N, K = (int(torch.randint(1, n, (1,), generator=g)) for n in (33, 3000, 5000))
    group = [32, 64, 128, 384][seed % 4]
    dtype = [BF, HF][seed % 2]
    w = weights(seed, (), N, K, group, seed % 3 == 0, dtype, slack=seed % 2)
    x = rand(seed + 1, M, K, dtype=dtype)
    got = ptc.matmul_a16_s4(x, matrix(w))
    check(got, x, w, dtype)
    assert torch.equal(ptc.matmul_a16_s4(x, matrix(w)), got)
