"""The mixture-of-experts layer against a loop over experts in 64 bits, and with its neighbours."""
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
    assert ptc.gemm_poll_device_error() == ptc.PTC_OK


def layer(seed, T, D, I, E, k, group=128, zeros=False, dtype=BF, st=None, router_dtype=None):
    """x, router and the two weights (scales of the size that keeps h near 1)."""
    gu, dn = weights(seed, (E,), 2 * I, D, group, zeros, st or dtype), weights(seed + 1, (E,), D, I, group, zeros, st or dtype)
    for w, n in ((gu, D), (dn, I)):
        f = 2.0 ** -round(n ** 0.5).bit_length()  # (exact)
        w["scales"] = w["scales"] * f
        w["values"], w["size"] = w["values"] * f, w["size"] * f
    return dict(x=rand(seed + 2, T, D, dtype=dtype), router=rand(seed + 3, E, D, dtype=router_dtype or dtype, size=D ** -0.5),
                gu=gu, dn=dn, k=k, renormalize=bool(seed % 2))


def run(L, **kw):
    return ptc.moe_a16_s4(L["x"], L["router"], matrix(L["gu"]), matrix(L["dn"]), L["k"], renormalize=L["renormalize"],
                          return_routing=True, **kw)


def compare(L, got):
    """Errors, with m = 2^-17: gate and up within m of their products' sizes; silu's slope is at most 1.1 and its own
    rounding 2^-21; h keeps 22 bits, with bfloat16 tokens 11 (half a step, 2^-12), and 2^-24 of the largest of 128; down again m of the products' sizes; p is within the logits' FP32 sums, 2^-18 of
    their products' sizes each."""
    y, ids, p = got
    x, dtype, k = L["x"].double(), L["x"].dtype, L["k"]
    logits = x @ L["router"].double().t()
    # The kernel's choice is checked, then used: logits in falling order, none left out above the last (2^-18 apart is a tie).
    order = ids.long()
    assert ids.dtype == torch.int32 and bool(((order >= 0) & (order < logits.shape[1])).all())
    top = torch.gather(logits, 1, order)
    near = 2.0 ** -18 * (x.abs() @ L["router"].double().abs().t()).amax(-1, keepdim=True)
    assert bool((top[:, 1:] <= top[:, :-1] + near).all())
    rest = logits.scatter(1, order, float("-inf"))
    assert int((rest == float("-inf")).sum()) == order.numel() and bool((rest <= top[:, -1:] + near).all())
    e = torch.exp(top - top[:, :1])
    want_p = e / (e if L["renormalize"] else torch.exp(logits - top[:, :1])).sum(-1, keepdim=True)
    assert p.dtype == torch.float32 and bool(((p.double() - want_p).abs() <= (2 * near + 2.0 ** -18) * want_p).all())
    I, m = L["dn"]["K"], 2.0 ** -17
    want, bound, total = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x)
    for ex in range(logits.shape[1]):
        tok, slot = torch.nonzero(order == ex, as_tuple=True)
        if tok.numel() == 0:
            continue
        gu, size = x[tok] @ L["gu"]["values"][ex].t(), x[tok].abs() @ L["gu"]["size"][ex].t()
        g, u, sg, su = gu[:, :I], gu[:, I:], size[:, :I], size[:, I:]
        silu = g * torch.sigmoid(g)
        h = silu * u
        dh = m * (1.1 * sg * u.abs() + silu.abs() * su) + (2.0 ** -12 if dtype == BF else 2.0 ** -20) * h.abs() + m * m * sg * su
        near_max = torch.nn.functional.pad(h.abs(), (0, -I % 128)).view(len(tok), -1, 128).amax(-1)
        dh = dh + 2.0 ** -24 * near_max.repeat_interleave(128, 1)[:, :I]
        w = want_p[tok, slot].unsqueeze(1)
        want.index_add_(0, tok, w * (h @ L["dn"]["values"][ex].t()))
        total.index_add_(0, tok, w * (h @ L["dn"]["values"][ex].t()).abs())
        bound.index_add_(0, tok, w * (dh @ L["dn"]["values"][ex].abs().t() + m * (h.abs() @ L["dn"]["size"][ex].t())))
    eps = torch.finfo(dtype)
    bound = bound * (1 + 2 * near) + eps.eps / 2 * want.abs() + (2.0 ** -17 + 2 * near) * total + eps.smallest_normal * eps.eps
    assert y.dtype == dtype and y.shape == want.shape
    off = (y.double() - want).abs()
    assert bool((off <= bound).all()), (off / bound).max()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("group", [32, 64, 128, 256])
@pytest.mark.parametrize("T, D, I, E, k", [(1, 32, 16, 2, 1), (1, 256, 128, 8, 2), (2, 1, 1, 3, 3), (7, 1000, 333, 13, 3),
                                           (16, 130, 49, 5, 5), (9, 640, 96, 1, 1), (33, 200, 150, 20, 4), (64, 264, 72, 6, 2)])
def test_sizes(T, D, I, E, k, group, dtype):
    L = layer(T + D + k, T, D, I, E, k, group, group in (32, 128), dtype)
    compare(L, run(L))


@pytest.mark.parametrize("T, D, I, E, k", [(1, 2048, 1024, 64, 8), (4, 2048, 768, 128, 8), (16, 4096, 512, 8, 2), (64, 512, 256, 512, 8),
                                           (16, 512, 1024, 40, 32), (3, 5000, 640, 16, 4)])
def test_larger(T, D, I, E, k):
    L = layer(3 + T, T, D, I, E, k, 128, False, BF)
    compare(L, run(L))


@pytest.mark.parametrize("dtype, st, rt", [(BF, HF, torch.float32), (HF, BF, torch.float32), (HF, HF, HF)])
def test_types(dtype, st, rt):
    L = layer(50, 5, 300, 200, 9, 2, 64, True, dtype, st, rt)
    compare(L, run(L))


@pytest.mark.parametrize("zero_gate, zero_down", [(True, False), (False, True)])
def test_zeros_of_one_matrix(zero_gate, zero_down):
    L = layer(60, 5, 256, 128, 6, 2, 32, False, BF)
    other = layer(60, 5, 256, 128, 6, 2, 32, True, BF)
    L["gu"] = other["gu"] if zero_gate else L["gu"]
    L["dn"] = other["dn"] if zero_down else L["dn"]
    compare(L, run(L))


def test_every_token_to_one_expert():
    """An expert with all tokens (tiles of eight of them) beside experts with none."""
    for T in (8, 9, 31, 64):
        L = layer(70, T, 384, 96, 12, 2, 128, False, BF)
        L["x"][:, 0] = 4.0
        L["router"][:, 0] = 0
        L["router"][7, 0] = 16.0
        got = run(L)
        assert bool((got[1][:, 0] == 7).all())
        compare(L, got)


def test_ties_go_to_the_lowest():
    L = layer(80, 6, 128, 32, 40, 5, 32, False, HF)
    L["router"][:] = 0
    y, ids, p = run(L)
    assert torch.equal(ids, torch.arange(5, device=DEV, dtype=torch.int32).expand(6, 5))
    assert torch.allclose(p, torch.full_like(p, 0.2 if L["renormalize"] else 1 / 40), rtol=2.0 ** -20)
    L["router"][33] = L["router"][4] = L["x"][0] / 64
    ids = run(L)[1]
    assert ids[0].tolist() == [4, 33, 0, 1, 2]


def test_logits_that_are_not_finite():
    """NaN counts as the smallest; every expert that is chosen exists; other tokens do not change."""
    L = layer(91, 9, 256, 64, 20, 3, 64, False, BF)
    clean = run(L)
    L["x"][2, 5] = float("nan")
    L["x"][6, 7] = float("inf")
    y, ids, p = run(L)
    keep = [0, 1, 3, 4, 5, 7, 8]
    assert torch.equal(y[keep], clean[0][keep]) and torch.equal(ids[keep], clean[1][keep]) and torch.equal(p[keep], clean[2][keep])
    assert ids[2].tolist() == [0, 1, 2] and bool(y[[2, 6]].isnan().all()) and bool(((ids >= 0) & (ids < 20)).all())
    L = layer(91, 4, 256, 64, 20, 3, 64, False, BF)
    L["router"][int(run(L)[1][0, 0])] = float("nan")
    ids, p = run(L)[1:]
    assert bool(ids[0, 0] >= 0) and (bool(p.isfinite().all()) if L["renormalize"] else True)


def test_large_values_of_h():
    """h far beyond binary16, and far below its smallest numbers."""
    for up in (2.0 ** 20, 2.0 ** -40):
        L = layer(101, 6, 256, 128, 4, 2, 128, False, BF)
        L["gu"]["scales"][:, 128:] *= up
        L["gu"]["values"][:, 128:] *= up
        L["gu"]["size"][:, 128:] *= up
        compare(L, run(L))


def test_views_and_out():
    L = layer(111, 5, 300, 130, 7, 2, 64, True, BF)
    want = run(L)
    buf = torch.full((5, 1000), 3.0, device=DEV, dtype=BF)
    buf[:, 7:307] = L["x"]
    L["x"] = buf[:, 7:307]
    out = buf[:, 501:801]
    got = run(L, out=out)
    assert got[0] is out
    compare(L, got)
    assert bool((buf[:, 307:501] == 3).all()) and bool((buf[:, 801:] == 3).all())
    one = ptc.moe_a16_s4(L["x"], L["router"], matrix(L["gu"]), matrix(L["dn"]), 2, renormalize=L["renormalize"])
    assert torch.equal(one, got[0]) and torch.equal(got[1], want[1])
    wide = torch.zeros(7, 700, 512, device=DEV, dtype=torch.uint8)
    w = L["gu"]["codes"].shape[2]
    wide[:, 100:360, 256:256 + w] = L["gu"]["codes"]
    S = ptc.S4Matrix.tile_scales
    gu = ptc.S4Matrix(wide[:, 100:360, 256:256 + w], S(L["gu"]["scales"]), 300, 64, S(L["gu"]["zeros"]))
    assert torch.equal(ptc.moe_a16_s4(L["x"], L["router"], gu, matrix(L["dn"]), 2, renormalize=L["renormalize"]), got[0])


def test_no_tokens():
    L = layer(121, 3, 128, 64, 4, 2)
    L["x"] = L["x"][:0]
    y, ids, p = run(L)
    assert y.shape == (0, 128) and ids.shape == p.shape == (0, 2)


@pytest.mark.parametrize("seed", range(10))
def test_random_sizes(seed):
    g = torch.Generator().manual_seed(seed)
    T, D, I, E, k = (int(torch.randint(1, n, (1,), generator=g)) for n in (40, 900, 500, 60, 9))
    L = layer(200 + seed, T, D, I, E, min(k, E), [32, 64, 128, 256][seed % 4], seed % 3 == 0, [BF, HF][seed % 2])
    got = run(L)
    compare(L, got)
    for a, b in zip(run(L), got):
        assert torch.equal(a, b)


def test_calls_at_once():
    """Calls on two streams, each with a workspace of its own, as from one."""
    A, B = layer(131, 4, 1024, 512, 16, 4), layer(141, 16, 512, 256, 32, 4)
    args = [(L["x"], L["router"], matrix(L["gu"]), matrix(L["dn"]), 4) for L in (A, B)]
    want = [ptc.moe_a16_s4(*a) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            got[i].append(ptc.moe_a16_s4(*args[i], stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, want[i]) for g in got[i])


def test_graph():
    """A captured layer, replayed with other tokens, and two graphs in turn."""
    A, B = layer(151, 4, 512, 256, 16, 4), layer(161, 9, 512, 256, 16, 2)
    graphs, outs, want = [], [], []
    for L in (A, B):
        m = matrix(L["gu"]), matrix(L["dn"])
        want.append(ptc.moe_a16_s4(L["x"], L["router"], *m, L["k"]))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(ptc.moe_a16_s4(L["x"], L["router"], *m, L["k"]))
        graphs.append((g, m))
    keep = A["x"].clone()
    for _ in range(3):
        A["x"].copy_(rand(9, 4, 512, dtype=BF))
        graphs[0][0].replay()
        graphs[1][0].replay()
        assert torch.equal(outs[1], want[1]) and not torch.equal(outs[0], want[0])
        A["x"].copy_(keep)
        graphs[0][0].replay()
        assert torch.equal(outs[0], want[0])


def test_a_wait_that_runs_out_is_reported():
    """An item that is never reported done: the waits end, the status says so, and the next call is whole."""
    L = layer(171, 4, 512, 256, 16, 4)
    want = run(L)
    torch.cuda.synchronize()
    ptc.ptc_debug_set_wait_limit(20_000_000, 3)
    try:
        run(L)
        torch.cuda.synchronize()
        assert ptc.lib().gemm_poll_device_error() == ptc.PTC_ERR_TIMEOUT
    finally:
        ptc.ptc_debug_set_wait_limit(0, -1)
    for a, b in zip(run(L), want):
        assert torch.equal(a, b)


def test_a_block_of_a_quantised_model():
    """The operators as a decoding step uses them: norm with the residual, a product, the norm in 8 bits for the INT8
    product, norm, experts; each against 64 bits from what it was given."""
    T, D = 6, 512
    L = layer(181, T, D, 256, 8, 2, 128, False, BF)
    wo = weights(182, (), D, D, 128, True, BF)
    x, res, g = rand(183, T, D, dtype=BF), rand(184, T, D, dtype=BF), rand(185, D, dtype=BF)
    y, s = ptc.rms_norm(x, g, residual=res)
    o = ptc.matmul_a16_s4(y, matrix(wo))
    check(o, y, wo, BF)
    q, scale, s2 = ptc.rms_norm_s8(o, g, residual=s)
    w8 = torch.randint(-127, 128, (D, D), generator=gen(186), device=DEV).to(torch.int8)
    z = ptc.matmul_s8_scaled(q, w8, scale, out_dtype=BF)
    n = ptc.rms_norm(z, g)
    L["x"] = n
    compare(L, run(L))
    assert torch.equal(s2, (o.float() + s.float()).to(BF))


def test_refusals():
    L = layer(191, 4, 256, 128, 6, 2)
    gu, dn, x, r = matrix(L["gu"]), matrix(L["dn"]), L["x"], L["router"]
    S = ptc.S4Matrix.tile_scales
    many = rand(1, 64, 256, dtype=BF)
    bad = [
        (TypeError, lambda: ptc.moe_a16_s4(x.float(), r, gu, dn, 2)), (TypeError, lambda: ptc.moe_a16_s4(x, r.half(), gu, dn, 2)),
        (ValueError, lambda: ptc.moe_a16_s4(x, r[:5], gu, dn, 2)), (ValueError, lambda: ptc.moe_a16_s4(x, r, dn, gu, 2)),
        (ValueError, lambda: ptc.moe_a16_s4(x[:, :128], r, gu, dn, 2)), (TypeError, lambda: ptc.moe_a16_s4(x, r, gu.codes, dn, 2)),
        (ptc.PtcError, lambda: ptc.moe_a16_s4(x, r, gu, dn, 0)), (ptc.PtcError, lambda: ptc.moe_a16_s4(x, r, gu, dn, 7)),
        (ptc.PtcError, lambda: ptc.moe_a16_s4(x, r, gu, dn, -1)), (ptc.PtcError, lambda: ptc.moe_a16_s4(x, r, gu, dn, 2, out=x)),
        (ptc.PtcError, lambda: ptc.moe_a16_s4(torch.cat([many, x]), r, gu, dn, 2)),
        (ValueError, lambda: ptc.moe_a16_s4(x, r, gu, ptc.S4Matrix(dn.codes, dn.scales.half(), 128), 2)),
        (ValueError, lambda: ptc.moe_a16_s4(x, r, gu, ptc.S4Matrix(dn.codes, dn.scales, 128, 256), 2)),
        (ValueError, lambda: ptc.moe_a16_s4(x, r, ptc.S4Matrix(gu.codes[0], gu.scales, 256), dn, 2)),
        (ValueError, lambda: ptc.moe_a16_s4(x, r, gu, dn, 2, out=x.half())), (ValueError, lambda: ptc.moe_a16_s4(x, r.cpu(), gu, dn, 2)),
        (RuntimeError, lambda: ptc.moe_a16_s4(x.clone().requires_grad_(), r, gu, dn, 2)),
        (RuntimeError, lambda: ptc.moe_a16_s4(x, r.clone().requires_grad_(), gu, dn, 2)),
    ]
    for error, call in bad:
        with pytest.raises(error):
            call()
