"""Chunk attention with CTAs that walk many tiles: the packed ring goes round, key and value stages are
reused, references move between tiles, two streams alternate; in every width, head dim and kernel.

(With the automatic splits a small batch leaves a CTA one tile or two.)"""
import numpy as np
import pytest
import torch

from test_gpu_seq_ops import KERNELS, Twin, check_chunk, config

pytestmark = pytest.mark.gpu

# new tokens whose 4 T query rows a kv head select: the few-row kernel (12 rows; past fp16 caches and
# d_k 64, which it is not built for), the narrow one (16 and 32), one 128-row tile (two streams on
# alternate tiles), two row tiles (with a second block of rows)
TOKENS = (3, 4, 8, 30, 70)


def long_cache(**kw):
    return config(batch=1, n_q_heads=4, n_kv_heads=1, max_context=2400, **kw)


@pytest.mark.parametrize("kb,vb", [(8, 8), (8, 4), (4, 8), (8, 2), (2, 8), (2, 2), (2, 4), (4, 2), (4, 4), (16, 16)])
def test_chunk_many_tiles_of_every_width(kb, vb):
    tw = Twin(long_cache(k_bits=kb, v_bits=vb), [2175], seed=kb + vb)
    for T in TOKENS:
        check_chunk(tw, T, splits=(1, 2), kernels=KERNELS[:1])


@pytest.mark.parametrize("dk,kb,vb", [(32, 4, 2), (32, 2, 4), (32, 8, 8), (32, 16, 16), (64, 4, 2), (64, 2, 2), (64, 8, 8),
                                      (64, 16, 16)])
def test_chunk_many_tiles_of_every_head_dim(dk, kb, vb):
    tw = Twin(long_cache(d_k=dk, k_bits=kb, v_bits=vb), [2175], seed=dk + kb)
    for T in TOKENS:
        check_chunk(tw, T, splits=(1, 2), kernels=KERNELS[:1])


@pytest.mark.parametrize("gk,gv,R,ret", [(32, 32, 64, 0), (32, 128, 0, 1), (128, 32, 5, 1), (64, 64, 300, 1), (128, 128, 129, 0)])
@pytest.mark.parametrize("paged", [0, 1])
def test_chunk_many_tiles_of_groups_and_pages(gk, gv, R, ret, paged):
    """Prefixes that end inside a tile of 128, one to four pages a tile, lists of several tiles."""
    tw = Twin(long_cache(group_k=gk, group_v=gv, window=R, log_retain=ret, paged=paged), [2111], seed=gk + R)
    for T in TOKENS:
        check_chunk(tw, T, splits=(1, 2), kernels=KERNELS[:1])


def test_chunk_many_tiles_with_references_that_move():
    """Keys that grow along the cache: every tile's scores pass the reference of the ones before."""
    for kb, vb in ((4, 2), (16, 16)):
        tw = Twin(long_cache(k_bits=kb, v_bits=vb), [0], seed=kb)
        k, v = tw.tokens(2100)
        k = (k.astype(np.float64) * np.linspace(0.1, 6.0, 2100)[None, :, None]).astype(np.float16)
        tw.gc.prefill_sequence(0, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda())
        tw.oc[0] = tw.oracle()
        tw.oc[0].prefill(k[None], v[None])
        for T in TOKENS:
            check_chunk(tw, T, splits=(1,), kernels=KERNELS[:1])


@pytest.mark.parametrize("n_q,n_kv", [(2, 2), (4, 2), (16, 2), (3, 1)])
def test_chunk_query_groups_in_few_splits(n_q, n_kv):
    tw = Twin(config(n_q_heads=n_q, n_kv_heads=n_kv), [600, 850, 329], seed=n_q)
    for T in (7, 50, 140):
        check_chunk(tw, T, splits=(1, 2), kernels=KERNELS[:1])


def test_chunk_of_a_prompt_in_one_split():
    """Several tiles of new tokens behind the cache, causal and masked, in one CTA a row block."""
    tw = Twin(config(batch=1, n_q_heads=4, n_kv_heads=1, window=64), [500], seed=2)
    check_chunk(tw, 290, splits=(1, 2), kernels=KERNELS[:1])
    rng = np.random.default_rng(3)
    check_chunk(tw, 290, sees=[rng.random((290, 290)) < 0.5], splits=(1, 2), kernels=KERNELS[:1])
