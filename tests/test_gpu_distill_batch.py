"""Distillation of whole training batches on the GPU: from 512 rows on a row has half the threads, and forms of its own by
the vocabulary's size, against plain fp64."""
import pytest
import torch

pytestmark = pytest.mark.gpu

tj2 = pytest.importorskip("bit_fully_quantized_amd")

from test_gpu_losses import INF, NAN, distill_check, gen  # noqa: E402


def batch_inputs(T, V, k, dtype, seed, pitch=None):
    g = gen(seed)
    z = torch.randn(T, pitch or V, generator=g, device="cuda") * 3
    start = torch.randint(0, V, (T, 1), generator=g, device="cuda")
    step = torch.randint(1, max(2, V // k), (T, 1), generator=g, device="cuda")
    ids = (start + step * torch.arange(k, device="cuda")) % V
    drop = torch.rand(T, k, generator=g, device="cuda") < 0.2
    u = torch.randn(T, k, generator=g, device="cuda") * 2 + 5
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    y[torch.rand(T, generator=g, device="cuda") < 0.1] = -100
    w = torch.randn(T, generator=g, device="cuda")
    return z.to(dtype)[:, :V], torch.where(drop, -1, ids).int(), u.to(dtype), y, w


BF16, F32 = torch.bfloat16, torch.float32


# a row of 16-byte vectors by 512 threads: up to 4, 8, 13 and 26 in registers, and read again from memory
@pytest.mark.parametrize("dtype,V", [(BF16, 1000), (BF16, 9001), (BF16, 30001), (BF16, 50304), (BF16, 90001), (BF16, 120001),
                                     (F32, 777), (F32, 5001), (F32, 15001), (F32, 25001), (F32, 50001), (F32, 60001)])
@pytest.mark.parametrize("alpha", [1.0, 0.5])
def test_distill_batch(dtype, V, alpha):
    z, ids, u, y, w = batch_inputs(515, V, 40, dtype, V)
    distill_check(z, ids, u, 2.0, alpha, y, w)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("alpha", [1.0, 0.3])
def test_distill_batch_of_most_entries(dtype, alpha):
    """512 kept entries: one for each thread of a row."""
    z, ids, u, y, w = batch_inputs(530, 6000, 512, dtype, 3)
    y[:100] = ids[:100, 0].clamp(min=0)  # hard targets among the teacher's
    ids[50:60, 1] = ids[50:60, 0]        # an entry listed twice
    distill_check(z, ids, u, 1.5, alpha, y, w)


@pytest.mark.parametrize("dtype,V", [(BF16, 32003), (F32, 10007)])
def test_distill_rows_on_both_sides_of_a_batch(dtype, V):
    z, ids, u, y, w = batch_inputs(512, V, 30, dtype, 5)
    for T in (511, 512):
        distill_check(z[:T], ids[:T].contiguous(), u[:T].contiguous(), 2.0, 0.5, y[:T].contiguous(), w[:T].contiguous())


@pytest.mark.parametrize("dtype,V,pitch", [(BF16, 9001, 9003), (BF16, 53000, 53001), (BF16, 110001, 110003), (F32, 5001, 5002),
                                           (F32, 26001, 26003), (F32, 54001, 54003)])
def test_distill_batch_pitches_in_place_and_misaligned_output(dtype, V, pitch):
    T = 512
    z, ids, u, y, w = batch_inputs(T, V, 20, dtype, V, pitch)
    loss, dz = distill_check(z, ids, u, 2.0, 0.3, y, w)
    out = torch.full((T, V + 7), 9.0, device="cuda", dtype=dtype)
    opt = dict(temperature=2.0, alpha=0.3, targets=y, weight=w)
    _, d2 = tj2.distill_topk(z, ids, u, dlogits=out[:, 5:5 + V], **opt)
    assert torch.equal(d2, dz) and (out[:, :5] == 9).all() and (out[:, 5 + V:] == 9).all()
    buf = torch.empty_strided(z.shape, z.stride(), dtype=dtype, device="cuda").copy_(z)
    l3, d3 = tj2.distill_topk(buf, ids, u, dlogits=buf, **opt)
    assert d3 is buf and torch.equal(d3, dz) and torch.equal(l3, loss)


def test_distill_batch_special_rows():
    for dtype in (BF16, F32):
        z, ids, u, y, w = batch_inputs(600, 2001, 7, dtype, 9)
        ids[0] = -1                # the teacher kept nothing
        ids[1] = ids[1, 0].abs()   # one entry, listed again and again
        z[2, 100:900] = -INF       # masked logits that nobody names
        ids[2] = torch.arange(7, device="cuda", dtype=torch.int32)
        y[2] = 5
        z[3] = NAN                 # ignored, whatever it holds
        y[3] = -100
        for alpha in (1.0, 0.4):
            loss, dz = distill_check(z, ids, u, 2.0, alpha, y, w)
            assert loss[3] == 0 and (dz[3] == 0).all() and (dz[2, 100:900] == 0).all()
