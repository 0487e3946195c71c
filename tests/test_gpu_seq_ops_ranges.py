"""Chunk attention where the values are small, where a CTA walks many tiles, and where calls are
padded or long: what the split and row-block plans do there, and the workspace they ask for."""
import ctypes

import numpy as np
import pytest
import torch

from mixed_precision_quantized_pack_b200 import kvq as K
import test_gpu_seq_ops as seq_ops
from test_gpu_seq_ops import KERNELS, VAR, Twin, check_chunk, config

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _reference_of_no_rows(monkeypatch):
    """The plain form of a sequence without new tokens: no rows (its side-code term takes one at least)."""
    full = seq_ops.reference

    def reference(tw, b, q, k_new, v_new, sees):
        if q.shape[1] == 0:
            empty = np.zeros(q.shape[:2] + (tw.cfg["d_v"],))
            return empty, empty
        return full(tw, b, q, k_new, v_new, sees)
    monkeypatch.setattr(seq_ops, "reference", reference)


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


@pytest.mark.parametrize("T,counts,masked", [(200, [200, 131, 7], False), (90, [90, 0, 89], True), (17, [17, 1, 16], False)])
def test_chunk_side_code_prompts(T, counts, masked):
    """Many row blocks over a side code: blocks that see few of the new tokens, blocks of rows behind
    the valid ones, blocks across two heads, an empty cache."""
    tw = Twin(config(side_rank=4, side_bits=4), [0, 640, 300], seed=T)
    sees = None
    if masked:
        rng = np.random.default_rng(T)
        sees = [rng.random((T, T)) < 0.2 for _ in range(3)]
    check_chunk(tw, T, counts=counts, sees=sees, splits=(0, 1, 3), kernels=KERNELS[:1])
    check_chunk(Twin(config(side_rank=8, side_bits=4, n_q_heads=2), [129, 0, 5], seed=T), T, counts=counts, sees=sees,
                kernels=KERNELS[:1])


@pytest.mark.parametrize("kb", [2, 4])
@pytest.mark.parametrize("rank,bits", [(4, 4), (4, 8), (8, 4)])
def test_chunk_side_code_up_to_24_rows(kb, rank, bits):
    """17 to 24 query rows over a side code: two blocks of rows for a few sequences, one for more."""
    for batch, lengths in ((3, [700, 129, 400]), (13, [300, 130, 0, 513] + [200 + 7 * i for i in range(9)])):
        tw = Twin(config(batch=batch, side_rank=rank, side_bits=bits, k_bits=kb), lengths, seed=batch)
        for T in (5, 6):
            check_chunk(tw, T, splits=(0, 1), kernels=KERNELS[:1])


def test_chunk_workspace_is_linear_in_the_new_tokens():
    """Two partials a row and no more once the rows fill the GPU, whatever stands in the cache; below
    that, what the splits of a few CTAs an SM leave."""
    for batch, L in ((1, 0), (1, 700), (8, 700), (2, 9000)):
        tw = Twin(config(batch=batch, n_q_heads=32, n_kv_heads=8, max_context=32768, side_rank=4, side_bits=4), [0] * batch)
        if L:
            k = torch.randn((batch, 8, L, 128), device="cuda").half()
            tw.gc.prefill(k, k)
        for T in (1, 4, 16, 100, 1024, 4096, 8192, 65536):
            for splits in (0, 8):
                partial = batch * 32 * T * (128 + 2) * 4
                size = K.kvq_chunk_workspace_size(tw.gc.handle, T, splits)
                assert size <= partial * max(2, splits + 1) + (32 << 20), (batch, L, T, splits, size)
        tw.gc.close()


def launches(call):
    """Graph nodes that a captured call leaves."""
    g = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(g):
        call()
    n = ctypes.c_size_t()
    assert ctypes.CDLL("libcuda.so.1").cuGraphGetNodes(ctypes.c_void_p(g.raw_cuda_graph()), None, ctypes.byref(n)) == 0
    return n.value


@pytest.mark.filterwarnings("ignore:The CUDA Graph is empty")
@pytest.mark.parametrize("extra", [VAR, dict(), dict(side_rank=4, side_bits=4, rot_keys=1)])
def test_chunk_padding_is_not_worked_through(extra):
    """A chunk padded to more tokens than any sequence brings costs a width map no further passes over
    the cache, and one without a token no launch at all."""
    tw = Twin(config(**extra), [640, 300, 513], seed=6)
    gc = tw.gc
    gc.set_kernel(K.KVQ_KERNEL_TENSOR)

    def count(T, counts):
        q, k, v = [torch.from_numpy(x).cuda() for x in tw.chunk(T)]
        out = torch.zeros((3, 8, T, 128), dtype=torch.float16, device="cuda")
        return launches(lambda: gc.chunk_attention(q, k, v, counts=counts, out=out))
    assert count(40, [0, 0, 0]) == 0
    assert count(40, [3, 0, 2]) <= count(3, [3, 0, 2]) + 1          # (one more to reorder the queries)
    assert count(40, [18, 0, 2]) <= count(18, [18, 0, 2]) + 1
    check_chunk(tw, 40, counts=[18, 0, 2], kernels=(K.KVQ_KERNEL_TENSOR,))
    check_chunk(tw, 40, counts=[3, 1, 2], kernels=(K.KVQ_KERNEL_TENSOR,))


@pytest.mark.parametrize("extra", [dict(), dict(k_bits=2), dict(v_bits=4), dict(k_bits=8, v_bits=4), dict(d_k=32),
                                   dict(group_k=32, group_v=32), dict(side_rank=4, side_bits=4),
                                   dict(side_rank=8, side_bits=4, rot_keys=1), dict(paged=1, n_q_heads=2)])
def test_chunk_of_up_to_four_rows_is_as_exact_as_a_decode(extra):
    """Up to four query rows of a kv head nothing but the output is rounded to 11 bits.

    The output's rounding is off by at most 2^-11 of an element and spread evenly over that, so its
    2-norm is at most 2^-11 / sqrt(3) = 2.8e-4 of the output's; halves of 11 bits each leave 2^-22 of
    a product, and MMAs that truncate fp32 sums at most 2^-22 a step over 4000 / 16 steps: 6e-5."""
    n_rep = extra.get("n_q_heads", 8) // 2
    for lengths in ([4000, 300, 1], [129, 0, 64]):
        tw = Twin(config(max_context=4096, **extra), lengths, seed=3)
        for T in (1, 2, 4):
            if n_rep * T > 4:
                continue
            check_chunk(tw, T, splits=(0, 1, 3), kernels=KERNELS[:1])
            q, k_new, v_new = tw.chunk(T)
            for ns in (0, 1):
                got = tw.gc.chunk_attention(*[torch.from_numpy(x).cuda() for x in (q, k_new, v_new)], num_splits=ns)
                got = got.double().cpu().numpy()
                for b in range(3):
                    ref, _ = seq_ops.reference(tw, b, q[b], k_new[b], v_new[b], seq_ops.causal(T))
                    err = np.linalg.norm(got[b] - ref) / np.linalg.norm(ref)
                    assert err <= 3.4e-4, (lengths, T, ns, b, err)
