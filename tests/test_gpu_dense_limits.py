"""smla_attend_dense at the ends of what its fp16 operands hold: latent scales around the last one whose
largest code stays finite.  Values are checked with the bounds that tests/test_gpu_dense.py derives."""
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
