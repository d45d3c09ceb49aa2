"""The largest scale of packed attention and of log probabilities: scale log2(e) has to be a number of fp32."""
import ctypes

import pytest
import torch

P = 0x10000  # a 16-byte aligned fake address: what reaches validation never launches
LARGEST = 2.35e38


@pytest.fixture(scope="module")
def L():
    from rank_bottleneck_block_gb300 import build

    build.build()
    from rank_bottleneck_block_gb300 import lowrank

    lowrank.lib()
    return lowrank


def _calls(L, scale):
    sh, big = L.lr_packed_shape(16, 2, 4, 2, 64), 1 << 30
    lib = L.lib()
    return (lib.lr_packed_attn_fwd(1, ctypes.byref(sh), scale, P, P, 256, P, 128, P, 128, P, 256, P, P, big, None),
            lib.lr_packed_attn_bwd(1, ctypes.byref(sh), scale, P, P, 256, P, 128, P, 128, P, 256, P, P, 256, P, 256, P, 128,
                                   P, 128, P, big, None),
            lib.lr_logprob_fwd(1, 4, 100, scale, 0, P, 100, P, P, P, P, None, None, P, big, None),
            lib.lr_logprob_bwd(1, 4, 100, scale, P, 100, P, P, P, P, P, P, 100, None))


@pytest.mark.parametrize("scale", [2.36e38, 3e38, 3.4e38])
def test_scales_beyond_are_refused(L, scale):
    assert _calls(L, scale) == (2, 2, 2, 2) and "scale" in L.lr_last_error()


def test_the_largest_is_taken(L):
    if torch.cuda.is_available():
        pytest.skip("a device is present: the calls would launch")
    assert _calls(L, LARGEST) == (8, 8, 8, 8)  # validated, but no device


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_log_probabilities_at_the_largest(L, dtype):
    """All weight on the largest logits, whatever else the row holds."""
    from rank_bottleneck_block_gb300 import inputs as I
    from rank_bottleneck_block_gb300.runner import TokenLogProbs

    shape = I.LogProbShape(T=3, V=5000, top=3, scale=LARGEST, dtype=dtype)
    case = I.make_logprob_case(shape, seed=1, entropy=False)
    z = case["logits"].clamp_(max=5.0)
    z[:, 7] = z[:, 4000] = 6.0
    case["target"] = torch.tensor([7, 4000, 7], dtype=torch.int32)
    case["dlogp"] = torch.full((3,), 2.0 ** -120)
    run = TokenLogProbs(shape, case)
    run.step()
    two = torch.full((3,), 2.0, dtype=torch.float64).log()
    assert ((run.logp.cpu().double() + two).abs() <= 1e-6).all() and ((run.entropy.cpu().double() - two).abs() <= 1e-6).all()
    assert (run.top_ids[:, :2].cpu() == torch.tensor([7, 4000])).all()
    want = torch.zeros(3, 5000, dtype=torch.float64)
    want[:, 7] = want[:, 4000] = -0.5 * 2.0 ** -120 * LARGEST
    want[torch.arange(3), case["target"].long()] *= -1
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -22
    assert ((run.dlogits.cpu().double() - want).abs() <= half * want.abs()).all()


@pytest.mark.gpu
def test_packed_attention_at_the_largest(L):
    """Equal scores (q is 0): every row the mean of the values it sees."""
    from rank_bottleneck_block_gb300 import inputs as I
    from rank_bottleneck_block_gb300.runner import PackedAttention

    shape = I.PackedShape(T=200, nseq=1, Hq=2, Hk=1, dh=64, scale=LARGEST)
    case = I.make_packed_case(shape, [200], seed=2)
    case["q"].zero_()
    run = PackedAttention(shape, case)
    run.forward()
    torch.cuda.synchronize()
    L.lr_check_device_error()
    v = case["v"].double()
    n = torch.arange(1, 201, dtype=torch.float64)[:, None]
    want, mag = v.cumsum(0) / n, v.abs().cumsum(0) / n
    for h in range(2):
        got = run.o[:, 64 * h:64 * h + 64].cpu().double()
        assert ((got - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -14) * mag).all()
    assert ((run.lse.cpu().double() - n.log()).abs() <= 1e-5).all()
