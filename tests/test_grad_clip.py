"""lr_grad_norm / lr_grad_clip on the GPU against fp64.

Bounds, u = 2^-24: fewer than 64 roundings on a square's way through the fp32 sums (32 in a row, the pairwise ones of
a warp) before the sum goes on in fp64: 65 u of the sum of squares, half of that in the norm, and u for its last
rounding: 34 u.  scale = max_norm / (norm + 1e-6) adds 3 u, the product one, and the output half a step of its type.
"""
import numpy as np
import pytest
import torch

import oracle.qk_oracle as Q
from oracle.compare import as64

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from rank_bottleneck_block_gb300 import build

    build.build()


def _grads(sizes, dtype=torch.float32, seed=0, scale=1.0):
    gen = torch.Generator()
    gen.manual_seed(seed)
    return [(torch.randn(n, generator=gen) * scale * (0.1 + i % 7)).to(dtype).cuda() for i, n in enumerate(sizes)]


def _check(grads, outs, clip, max_norm):
    host = [as64(g) for g in grads]
    norm, scale, want = Q.clip(host, max_norm)
    assert abs(float(clip.norm) - norm) <= 34 * U * norm
    assert abs(float(clip.scale) - scale) <= 38 * U * scale
    for g, o, w in zip(grads, outs, want):
        assert (np.abs(as64(o) - w) <= (HALF[o.dtype] + 40 * U) * np.abs(w) + 1e-40).all()


LISTS = [[1], [7], [8, 1, 3], [8192], [8191, 8193, 16384], [0, 5, 0, 0, 70001, 0], [1_000_003], [33] * 50,
         [65536] * 9 + [1] * 9, [2_500_000, 3, 40_000]]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sizes", LISTS, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("max_norm", [0.5, 1e9])
def test_clip_matches_fp64(sizes, dtype, max_norm):
    from rank_bottleneck_block_gb300.runner import GradClip

    grads = _grads(sizes, dtype)
    keep = [g.clone() for g in grads]
    outs = [torch.full_like(g, 3.0) for g in grads]
    c = GradClip(grads, max_norm, outs)
    c.clip()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(grads, keep))
    _check(keep, outs, c, max_norm)
    if max_norm == 1e9:
        assert float(c.scale) == 1.0 and all(torch.equal(a, b) for a, b in zip(outs, keep))
    inp = GradClip(grads, max_norm)
    inp.clip()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(grads, outs))  # in place: the same bits
    c2 = GradClip(keep, max_norm)
    c2.stat.fill_(-1.0)
    c2.measure()
    assert float(c2.norm) == float(c.norm) and float(c2.scale) == -1.0


def test_nothing_beside_the_tensors_is_written():
    """Tensors at 16-byte aligned places of one buffer, odd sizes: the gaps keep their values."""
    from rank_bottleneck_block_gb300.runner import GradClip

    for dtype, step in ((torch.float32, 4), (torch.bfloat16, 8)):
        sizes = [5, 1, 8193, 31, 20000, 3]
        flat = torch.full((40000,), 2.0, dtype=dtype, device="cuda")
        mask, at, views = torch.zeros(40000, dtype=torch.bool, device="cuda"), 16, []
        for n in sizes:
            views.append(flat[at:at + n])
            mask[at:at + n] = True
            at += (n + step) // step * step + 2 * step
        keep = [v.clone() for v in views]
        c = GradClip(views, 1.0)
        c.clip()
        assert (flat[~mask] == 2.0).all()
        _check(keep, views, c, 1.0)


def test_more_tensors_than_one_launch_takes():
    from rank_bottleneck_block_gb300.runner import GradClip

    grads = _grads([1 + (37 * i) % 300 for i in range(2500)])
    keep = [g.clone() for g in grads]
    c = GradClip(grads, 2.0)
    c.clip()
    _check(keep, grads, c, 2.0)
    empty = [torch.empty(0, device="cuda") for _ in range(1100)] + _grads([9])
    keep = [g.clone() for g in empty]
    c = GradClip(empty, 0.25)
    c.clip()
    _check(keep, empty, c, 0.25)


def test_lists_without_elements():
    from rank_bottleneck_block_gb300.runner import GradClip

    for n in (1, 16, 17, 300, 1500):
        c = GradClip([torch.empty(0, device="cuda") for _ in range(n)], 1.0)
        c.stat.fill_(-1.0)
        c.clip()
        assert float(c.norm) == 0.0 and float(c.scale) == 1.0


@pytest.mark.parametrize("n", [31 * 8192, 32 * 8192, 32 * 8192 + 1, 40 * 8192, 512 * 8192 + 5, 2100 * 8192])
def test_around_the_borders_of_the_kernels_choices(n):
    """One cluster up to 32 chunks of 32 KB, blocks that add the partial sums up themselves, a launch for that."""
    from rank_bottleneck_block_gb300.runner import GradClip

    for dtype, m in ((torch.float32, n), (torch.bfloat16, 2 * n)):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(n)
        g = torch.randn(m, generator=gen, device="cuda").to(dtype)
        out = torch.empty_like(g)
        c = GradClip([g[:m // 2 // 8 * 8], g[m // 2 // 8 * 8:]], 3.0, [out[:m // 2 // 8 * 8], out[m // 2 // 8 * 8:]])
        c.clip()
        norm = float(g.double().square().sum().sqrt())
        assert abs(float(c.norm) - norm) <= 34 * U * norm
        want = g.double() * (3.0 / (norm + 1e-6))
        assert ((out.double() - want).abs() <= (HALF[dtype] + 40 * U) * want.abs() + 1e-40).all()


def test_a_tensor_of_more_than_2_to_the_31_elements():
    from rank_bottleneck_block_gb300.runner import GradClip

    n = (1 << 31) + 12345
    g = torch.full((n,), 0.5, dtype=torch.bfloat16, device="cuda")
    g[-1] = 64.0
    c = GradClip([torch.ones(8, dtype=torch.bfloat16, device="cuda"), g], 1.0)
    c.clip()
    norm = (8 + (n - 1) * 0.25 + 4096.0) ** 0.5
    assert abs(float(c.norm) - norm) <= 34 * U * norm
    want = torch.tensor([0.5 / norm, 64.0 / norm], dtype=torch.float64)
    got = torch.stack([g[-2], g[-1]]).double().cpu()
    assert ((got - want).abs() <= (HALF[torch.bfloat16] + 40 * U) * want).all()
    assert (g[:-1] == g[0]).all()


@pytest.mark.parametrize("scale", [1e-30, 1e-22, 1e-19, 1e-18, 1e-17, 1e-16, 1e-14, 1e15, 1e18, 1e25, 1e37])
def test_squares_beyond_the_fp32_range_are_kept(scale):
    from rank_bottleneck_block_gb300.runner import GradClip

    grads = _grads([30000, 11], scale=scale / 10)
    keep = [g.clone() for g in grads]
    c = GradClip(grads, 1.0)
    c.measure()
    norm = Q.clip([as64(g) for g in keep], 1.0)[0]
    if norm < 3e38:
        assert abs(float(c.norm) - norm) <= 34 * U * norm
        c.clip()
        _check(keep, grads, c, 1.0)
    else:
        assert float(c.norm) == float("inf")


def test_scales_that_differ_by_forty_orders_of_magnitude():
    from rank_bottleneck_block_gb300.runner import GradClip

    grads = [torch.full((50000,), 1e-25, device="cuda"), torch.full((50000,), 1e20, device="cuda"),
             torch.zeros(50000, device="cuda"), torch.full((40000,), 1e-3, device="cuda")]
    grads[3][::1000] = 1e19
    c = GradClip(grads, 1.0)
    c.measure()
    norm = Q.clip([as64(g) for g in grads], 1.0)[0]
    assert abs(float(c.norm) - norm) <= 34 * U * norm


@pytest.mark.parametrize("low", [-17, -18, -19])
def test_squares_around_the_smallest_normal_number(low):
    """Elements from 10^low over six orders of magnitude upwards: many squares are fp32 denormals, few carry the sum."""
    from rank_bottleneck_block_gb300.runner import GradClip

    for top in (0.0, 1.0, 2.5, 6.0):
        gen = torch.Generator()
        gen.manual_seed(int(10 * top) - low)
        g = 10.0 ** (low + top * torch.rand(50000, generator=gen, dtype=torch.float64) ** 8)
        grads = [g.float().cuda()]
        c = GradClip(grads, 1.0)
        c.measure()
        norm = Q.clip([as64(grads[0])], 1.0)[0]
        assert abs(float(c.norm) - norm) <= 34 * U * norm


def test_zeros_and_a_bound_of_zero():
    from rank_bottleneck_block_gb300.runner import GradClip

    z = [torch.zeros(1000, device="cuda"), torch.empty(0, device="cuda")]
    c = GradClip(z, 1.0)
    c.clip()
    assert float(c.norm) == 0.0 and float(c.scale) == 1.0 and (z[0] == 0).all()
    c = GradClip([torch.empty(0, device="cuda")], 1.0)
    c.clip()
    assert float(c.norm) == 0.0 and float(c.scale) == 1.0
    g = _grads([300])
    c = GradClip(g, 0.0)
    c.clip()
    assert float(c.scale) == 0.0 and (g[0] == 0).all()


@pytest.mark.parametrize("bad,scale", [(float("nan"), float("nan")), (float("inf"), 0.0), (float("-inf"), 0.0)])
def test_what_is_not_finite_is_reported(bad, scale):
    from rank_bottleneck_block_gb300.runner import GradClip

    grads = _grads([20000, 50])
    grads[0][12345] = bad
    outs = [torch.empty_like(g) for g in grads]
    c = GradClip(grads, 1.0, outs)
    c.clip()
    assert np.isnan(float(c.norm)) if np.isnan(bad) else float(c.norm) == float("inf")
    assert np.array_equal([float(c.scale)], [scale], equal_nan=True)
    assert torch.isnan(outs[0][12345])  # NaN * scale, inf * 0
    rest = outs[0][:12345]
    assert torch.isnan(rest).all() if np.isnan(bad) else (rest == 0).all()


def test_repeats_bitwise_and_in_graphs_that_share_a_workspace():
    from rank_bottleneck_block_gb300.runner import GradClip, GraphStep

    grads = _grads([123457, 8, 999, 400000])
    outs = [torch.empty_like(g) for g in grads]
    c = GradClip(grads, 1.0, outs)
    c.clip()
    ref = [o.clone() for o in outs] + [c.stat.clone()]
    other = GradClip(_grads([5000, 70000], seed=4), 1.0, [torch.empty(n, device="cuda") for n in (5000, 70000)])
    other.clip()
    ref2 = [o.clone() for o in other.outs] + [other.stat.clone()]
    assert other.ws.numel() <= c.ws.numel()
    other.ws = c.ws  # replayed one after the other on one stream
    graphs = [GraphStep(c.clip), GraphStep(other.clip)]
    for _ in range(3):
        for t in outs + other.outs:
            t.zero_()
        for g in graphs:
            g()
        assert all(torch.equal(a, b) for a, b in zip(ref, outs + [c.stat]))
        assert all(torch.equal(a, b) for a, b in zip(ref2, other.outs + [other.stat]))


def test_the_mlp_block_clips_its_gradients():
    """Forward, backward and clipping of a block as a training step runs them."""
    from rank_bottleneck_block_gb300 import inputs as I
    from rank_bottleneck_block_gb300.runner import BlockStack, MlpBlock

    shape = I.MlpShape(T=128, d=256, f=688, r=64, dtype="f32")
    blk = MlpBlock(shape, I.make_mlp_case(shape, seed=0))
    blk.step()
    keep = [t.clone() for t in blk.grad_tensors()]
    norm = blk.clip_grads(1.0)
    assert len(keep) == 7 and float(norm) > 1.0
    _check(keep, blk.grad_tensors(), blk._clip, 1.0)
    stack = BlockStack(shape, I.make_stack_case(shape, 3, seed=1))
    stack.step()
    keep = [t.clone() for t in stack.grad_tensors()]
    stack.clip_grads(1e-3)
    assert len(keep) == 21
    _check(keep, stack.grad_tensors(), stack._clip, 1e-3)


def test_clipping_follows_replaced_gradients_and_covers_the_group():
    from rank_bottleneck_block_gb300 import inputs as I
    from rank_bottleneck_block_gb300.runner import MlpBlock, ProjGroup

    shape = I.MlpShape(T=128, d=256, f=688, r=64, dtype="f32")
    blk = MlpBlock(shape, I.make_mlp_case(shape, seed=0))
    blk.step()
    blk.clip_grads(1.0)
    blk.grads["dA_up"] = torch.empty_like(blk.grads["dA_up"])
    blk.step()
    keep = [t.clone() for t in blk.grad_tensors()]
    blk.clip_grads(1.0)
    _check(keep, blk.grad_tensors(), blk._clip, 1.0)
    shape = I.ProjShape(T=100, d_in=128, d_out=64, r=32, group=2)
    group = ProjGroup(shape, I.make_proj_case(shape, seed=1))
    group.step()
    keep = [t.clone() for t in group.grad_tensors()]
    assert len(keep) == 5
    group.clip_grads(0.5)
    _check(keep, group.grad_tensors(), group._clip, 0.5)
