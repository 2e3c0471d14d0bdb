"""smla_attend_dense at the ends of what its fp16 operands hold: latent scales around the last one whose
largest code stays finite, and scores of any size.  Values are checked with the bounds that tests/test_gpu_dense.py derives."""
import numpy as np
import pytest
import torch

import paged_sparse_mla_gb300 as smla
from tests import gpu_helpers as G
from tests.test_gpu_dense import Case, ok

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G.ensure_built()


def record(c, pos):
    """The 656 bytes of position `pos` of the first sequence."""
    return c.pool.view(-1, c.lay.block_stride)[int(c.table[0, pos // c.bs]), :c.bs * 656].view(c.bs, 656)[pos % c.bs]


END = 146.1875  # half way between fp16's 146.125 (x 448 = 65,464) and 146.25 (x 448 = 65,520, which fp16 rounds to infinity)


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("pos", [5, 70, 199])
@pytest.mark.parametrize("scale,latched", [(146.125, False), (146.18, False), (float(np.nextafter(np.float32(END), np.float32(0))), False),
                                           (END, True), (146.2, True), (65504 / 448, True), (146.25, True)])
def test_scales_up_to_the_last_finite_one(scale, latched, pos, sign):
    """A tile with code 448 of either sign is exact to fp16's roundings up to the last scale whose rounded value
    keeps it finite; from the first that does not, the call latches."""
    c = Case([200], [3], 64, seed=51, q_scale=1e-4)
    rec = record(c, pos)
    rec[384 + 9] = 0x7E                                   # +448 and -448 of the last tile
    rec[384 + 10] = 0xFE
    s = np.float32(sign * scale)
    rec[524:528] = torch.from_numpy(np.array([s])).cuda().view(torch.uint8)
    got = c.run()
    if latched:
        assert smla.smla_get_last_error() == 7
        return
    ok()
    lat, rope = c.keys[0][0].copy(), c.keys[0][1]
    lat[pos, 384:512] = rec[384:512].view(torch.float8_e4m3fn).double().cpu().numpy() * float(s)
    c.check(got, keys=[(lat, rope)])


@pytest.mark.parametrize("q_scale", [1e4, 1e5, 1e6, 1e8, 1e20])
def test_scores_beyond_fp32s_integers(q_scale):
    """Scores so large that neighbouring fp32 values are whole powers of two apart in probability: weights come from
    differences of scores, so that the outputs stay averages of the values."""
    c = Case([333, 65], [3, 1], 64, seed=10, key_scale=1e3, q_scale=q_scale)
    for workspace in (True, False):
        out, lse = c.run(workspace)
        ok()
        c.check((out, lse))
        assert torch.isfinite(lse).all()
        for row, (lat, _) in zip((0, 3), c.keys):
            assert out[row].abs().max() <= 1.01 * np.abs(lat).max()
    # one position whose score is the largest by far more than the keys' roundings takes everything
    c.q[:], c.q_pe[:] = 0, 0
    c.q_pe[..., 0] = q_scale
    slots = [int(c.table[b, j // 64]) for b, j in ((0, 100), (1, 30))]
    blocks = c.pool.view(-1, c.lay.block_stride)
    for blk, j in zip(slots, (100, 30)):
        blocks[blk, (j % 64) * 656 + 528:(j % 64) * 656 + 530] = torch.tensor([1e4], device="cuda").bfloat16().view(torch.uint8)
    for workspace in (True, False):
        out, _ = c.run(workspace)
        ok()
        for t, (lat, j) in enumerate(((c.keys[0][0], 100),) * 3 + ((c.keys[1][0], 30),)):
            want = torch.from_numpy(lat[j]).cuda()
            assert ((out[t].double() - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -10 + 2.0 ** -11) + 2.0 ** -25).all()
