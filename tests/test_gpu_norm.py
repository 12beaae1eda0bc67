"""GPU parity: residual addition, RMS norm and MXFP8 quantisation in one pass.

Tolerances, before any run: the sum is one fp32 addition of two bf16 values and one rounding, so it equals the
rounding of the exact sum except where fp32 rounded first: within one bf16 step, 2^-8 of its magnitude. The norm is
rounded to bf16 once (2^-8 / (1 + 2^-8) at most) after a handful of fp32 operations (each 2^-24, the sum of squares at most cols * 2^-24
relative): within 2^-8. Codes and scales equal the quantiser's on the rounded norm, bit for bit.
"""
import numpy as np
import pytest
import torch

from oracle import attention as A

pytestmark = pytest.mark.gpu
EPS = 1e-6


def _inputs(rows, cols, seed, residual=True):
    rng = np.random.default_rng(seed)
    ch = np.exp(rng.standard_normal(cols))
    bf = lambda a: torch.from_numpy(np.asarray(a, dtype=np.float32)).to(torch.bfloat16).cuda()  # noqa: E731
    x = bf(rng.standard_normal((rows, cols)) * ch)
    r = bf(3 * rng.standard_normal((rows, cols)) * ch) if residual else None
    return x, r, bf(1 + 0.1 * rng.standard_normal(cols))


def _np(t):
    return None if t is None else t.float().cpu().numpy().astype(np.float64)


def _check(x, r, w, y, total, q, s, eps=EPS):
    from block_scaled_fp8_moe_gb300 import binding as B
    h, want = A.add_rmsnorm(_np(x), _np(r), _np(w), eps)
    assert np.all(np.abs(_np(total) - h) <= 2.0 ** -8 * np.abs(h))
    assert np.all(np.abs(_np(y) - want) <= 2.0 ** -8 * np.abs(want) + 1e-38)
    if q is not None:
        rq, rs = B.moe_quant_mxfp8(y)
        assert torch.equal(q.view(rq.shape), rq) and torch.equal(s.view(rs.shape), rs)


@pytest.mark.parametrize("rows,cols", [(1, 32), (6, 4096), (3, 96), (17, 512), (9, 544), (5, 1056), (33, 2080),
                                       (4, 8224), (2, 16384), (300, 4096), (1, 16352)])
@pytest.mark.parametrize("residual", [True, False])
def test_norm_matches_the_oracle(rows, cols, residual):
    from block_scaled_fp8_moe_gb300 import binding as B
    x, r, w = _inputs(rows, cols, rows * 31 + cols, residual)
    x0 = x.clone()
    y, total, q, s = B.moe_add_rmsnorm_mxfp8(x, w, r, eps=EPS)
    _check(x, r, w, y, total, q, s)
    assert torch.equal(x, x0)


def test_zero_rows_tiny_and_huge_values():
    from block_scaled_fp8_moe_gb300 import binding as B
    x, r, w = _inputs(6, 256, 3)
    x[0] = 0
    r[0] = 0
    x[1] *= 1e-15
    r[1] *= 1e-15
    x[2] *= 1e15
    r[2] *= 1e15
    r[3] = -x[3]                        # the sum vanishes
    x[4, 7] = 3e4
    y, total, q, s = B.moe_add_rmsnorm_mxfp8(x, w, r, eps=EPS)
    _check(x, r, w, y, total, q, s)
    assert not y[0].any() and not y[3].any() and not s[0].any()
    y0 = B.moe_add_rmsnorm_mxfp8(x[1:3], w, r[1:3], eps=0.0)[0]
    _, want = A.add_rmsnorm(_np(x[1:3]), _np(r[1:3]), _np(w), 0.0)
    assert np.all(np.abs(_np(y0) - want) <= 2.0 ** -8 * np.abs(want))


def test_in_place_and_optional_outputs():
    from block_scaled_fp8_moe_gb300 import binding as B
    x, r, w = _inputs(70, 4096, 5)
    want = B.moe_add_rmsnorm_mxfp8(x, w, r)
    x1, r1 = x.clone(), r.clone()
    y, total, q, s = B.moe_add_rmsnorm_mxfp8(x1, w, r1, sum_out=r1, y=x1)
    assert total is r1 and y is x1
    for a, b in zip((y, total, q, s), want):
        assert torch.equal(a, b)
    y, total, q, s = B.moe_add_rmsnorm_mxfp8(x, w, r, quant=False)
    assert q is None and s is None and torch.equal(y, want[0]) and torch.equal(total, want[1])


def test_rows_do_not_depend_on_their_batch():
    from block_scaled_fp8_moe_gb300 import binding as B
    x, r, w = _inputs(301, 1536, 9)
    whole = B.moe_add_rmsnorm_mxfp8(x, w, r)
    for a, b in ((0, 1), (7, 9), (200, 301)):
        for p, q in zip(B.moe_add_rmsnorm_mxfp8(x[a:b].contiguous(), w, r[a:b].contiguous()), whole):
            assert torch.equal(p, q[a:b])


def test_a_value_that_is_not_finite_stays_in_its_row():
    from block_scaled_fp8_moe_gb300 import binding as B
    x, r, w = _inputs(40, 64, 11)
    want = B.moe_add_rmsnorm_mxfp8(x, w, r)
    x[3, 5] = float("nan")
    x[20, 5] = float("inf")
    y, total, q, s = B.moe_add_rmsnorm_mxfp8(x, w, r)
    keep = [i for i in range(40) if i not in (3, 20)]
    for a, b in zip((y, total, q, s), want):
        assert torch.equal(a[keep], b[keep])
    assert y[3].isnan().all() and y[20, 5].isnan() and not y[20, :5].any()


def test_feeds_the_layer_like_the_layers_own_quantisation():
    """Codes from the norm into the experts' products equal the layer's own call on the norm's bf16 rows."""
    from block_scaled_fp8_moe_gb300 import binding as B
    from block_scaled_fp8_moe_gb300 import synth
    cfg = synth.CONFIGS["tiny"]
    inp = synth.make_inputs_cpu(cfg)
    layer = B.MoeLayer.from_fp32(inp.w_router.cuda(), inp.bias.cuda(), inp.w13.cuda(), inp.w2.cuda(), cfg.k)
    x, r, w = _inputs(cfg.T, cfg.H, 1)
    y, _, q, s = B.moe_add_rmsnorm_mxfp8(x, w, r)
    shp, ws = layer.shape(cfg.T), layer.workspace(cfg.T)
    plan = B.moe_route_topk(shp, y, layer.w_router, layer.bias, None, ws)
    _, _, rows = B.moe_experts_grouped(shp, q, s, layer.w13p, layer.w13sp, layer.w2p, layer.w2sp, plan, ws)
    assert torch.equal(B.moe_combine(shp, rows, plan, ws), layer.forward(y))


def test_refusals():
    from block_scaled_fp8_moe_gb300 import binding as B
    x, r, w = _inputs(4, 64, 2)
    for call in (lambda: B.moe_add_rmsnorm_mxfp8(x.float(), w, r), lambda: B.moe_add_rmsnorm_mxfp8(x, w[:32], r),
                 lambda: B.moe_add_rmsnorm_mxfp8(x, w, r[:3]), lambda: B.moe_add_rmsnorm_mxfp8(x.t(), w, r),
                 lambda: B.moe_add_rmsnorm_mxfp8(x.cpu(), w, r),
                 lambda: B.moe_add_rmsnorm_mxfp8(x, w, r, y=torch.empty_like(x[:2]))):
        with pytest.raises(ValueError):
            call()
    for bad in (float("nan"), float("inf"), -1.0):
        with pytest.raises(B.MoeError):
            B.moe_add_rmsnorm_mxfp8(x, w, r, eps=bad)
    with pytest.raises(B.MoeError):
        B.moe_add_rmsnorm_mxfp8(x[:, :40].contiguous(), w[:40].contiguous())
    assert B.moe_add_rmsnorm_mxfp8(x[:0], w)[0].shape == (0, 64)


def test_residuals_of_other_shapes():
    """The rows in another number of dimensions are the same rows; the same elements in another order are not."""
    from block_scaled_fp8_moe_gb300 import binding as B
    x, r, w = _inputs(6, 64, 2)
    want = B.moe_add_rmsnorm_mxfp8(x, w, r)
    for a, b in ((x.view(2, 3, 64), r), (x, r.view(3, 2, 64)), (x, r.view(-1)), (x.view(2, 3, 64), r.view(2, 3, 64))):
        for p, q in zip(B.moe_add_rmsnorm_mxfp8(a, w, b), want):
            assert torch.equal(p.flatten(), q.flatten())
    for a, b in ((x, r.view(64, 6)), (x.view(2, 3, 64), r.view(3, 2, 64)), (x, r.view(3, 4, 32)), (x, r.view(12, 32))):
        with pytest.raises(ValueError, match="residual"):
            B.moe_add_rmsnorm_mxfp8(a, w, b)


def test_outputs_that_would_not_be_written_are_refused():
    from block_scaled_fp8_moe_gb300 import binding as B
    x, r, w = _inputs(6, 64, 2)
    q, s = torch.zeros(6, 64, dtype=torch.uint8, device="cuda"), torch.zeros(6, 2, dtype=torch.uint8, device="cuda")
    for kw in (dict(q=q), dict(s=s), dict(q=q, s=s)):
        with pytest.raises(ValueError):
            B.moe_add_rmsnorm_mxfp8(x, w, r, quant=False, **kw)
    assert B.moe_add_rmsnorm_mxfp8(x, w, r, q=q, s=s)[2] is q and q.any()
