"""Chunk attention where the values are small, where a CTA walks many tiles, and where calls are
padded or long: what the split and row-block plans do there, and the workspace they ask for."""
import numpy as np
import pytest
import torch

from mixed_precision_quantized_pack_b200 import kvq as K
from test_gpu_seq_ops import KERNELS, VAR, Twin, check_chunk, config

pytestmark = pytest.mark.gpu


class Scaled(Twin):
    """A twin whose values are `scale` times normal ones."""

    def __init__(self, cfg, lengths, scale, seed=0):
        self.scale = scale
        super().__init__(cfg, lengths, seed=seed)

    def tokens(self, n):
        k, v = super().tokens(n)
        return k, (v.astype(np.float64) * self.scale).astype(np.float16)


@pytest.mark.parametrize("extra", [dict(), dict(k_bits=2), dict(k_bits=8, v_bits=4, group_k=32, group_v=32),
                                   dict(side_rank=4, side_bits=4), dict(d_k=32, v_bits=4)])
@pytest.mark.parametrize("scale", [1e-4, 1e-5, 2e-6])
def test_chunk_small_values(extra, scale):
    """Values down to fp16's smallest: the elementwise bound has no term for products that vanish.

    Besides the output's own rounding (2^-25, in the bound) the few-row kernel adds no absolute
    error: a product of weight and value scale is exact to 2^-11 down to 2^-25 of the largest, and
    below that off by at most 2^-36 of it, over 4000 tokens less than 2^-24."""
    tw = Scaled(config(batch=1, max_context=4096, **extra), [4000], scale, seed=5)
    for T in (1, 4, 6):                    # 4, 16 and 24 query rows of a kv head
        check_chunk(tw, T, splits=(0, 1), kernels=KERNELS[:1])


def test_chunk_values_that_grow():
    """Value scales that grow and shrink along the cache by five orders of magnitude, in both
    directions: the few-row kernel's accumulators follow the largest."""
    need = config(batch=2, max_context=1024)
    for sign in (1, -1):
        tw = Twin(need, [0, 0], seed=17)
        for b, L in enumerate((1000, 640)):
            k, v = tw.tokens(L)
            size = 10.0 ** (sign * np.linspace(-2.5, 2.5, L))
            v = (v.astype(np.float64) * size[None, :, None]).astype(np.float16)
            tw.gc.prefill_sequence(b, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda())
            tw.oc[b] = tw.oracle()
            tw.oc[b].prefill(k[None], v[None])
        for T in (1, 4, 6):
            check_chunk(tw, T, splits=(0, 1, 3), kernels=KERNELS[:1])
