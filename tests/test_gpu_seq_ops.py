"""Chunk attention, multi-token append, forks and page compaction against plain forms.

Chunk attention is compared with fp64 attention over the oracle's decoded cache, element by
element, within a bound that is derived from the roundings the call makes (``chunk_bound``);
appends must leave the oracle's bytes; forks and compactions must not change a bit of what a
sequence holds.
"""
import math

import numpy as np
import pytest
import torch

from oracle import kvq_oracle as O
from mixed_precision_quantized_pack_b200 import kvq as K
from mixed_precision_quantized_pack_b200 import workloads as W
from test_gpu_parity import compare_state, need_gpu

pytestmark = pytest.mark.gpu
U16 = 2.0 ** -11          # half a step of fp16, relative
KERNELS = (K.KVQ_KERNEL_AUTO, K.KVQ_KERNEL_GENERIC)

BASE = dict(batch=3, n_q_heads=8, n_kv_heads=2, d_k=128, d_v=128, k_bits=4, v_bits=2, group_k=64, group_v=64,
            window=128, log_retain=1, max_context=1024)
VAR = dict(k_bits=0, v_bits=0, group_v=32, k_widths=[8] * 16 + [4] * 64 + [2] * 32 + [0] * 16,
           v_widths=[4] * 32 + [2] * 64 + [1] * 32)


def config(**kw):
    c = dict(BASE, **kw)
    if c.get("paged"):
        c.setdefault("n_pages", c["batch"] * -(-c["max_context"] // c["group_k"]) + 3)
    if c.get("rot_keys"):
        c.setdefault("rot_signs", W.rotation_signs(5))
    return c


class Twin:
    """A GPU cache and one oracle cache per sequence, fed the same tokens."""

    def __init__(self, cfg, lengths, seed=0):
        need_gpu()
        self.cfg, self.rng = cfg, np.random.default_rng(seed)
        H, dk, dv, r = cfg["n_kv_heads"], cfg["d_k"], cfg["d_v"], cfg.get("side_rank", 0)
        self.sigma = np.exp(self.rng.uniform(math.log(0.5), math.log(4.0), (H, 1, dk)))
        self.mu = self.rng.normal(0, 1, (H, 1, dk))
        self.basis = None
        if r:
            self.basis = np.linalg.qr(self.rng.normal(size=(H, dk, r)))[0].astype(np.float32)
        self.gc = K.KVCache(cfg, side_basis=None if self.basis is None else torch.from_numpy(self.basis))
        self.oc = [None] * cfg["batch"]
        for b, L in enumerate(lengths):
            if L:
                self.prefill(b, L)

    def oracle(self):
        return O.OracleCache(dict(self.cfg, batch=1), side_basis=self.basis)

    def tokens(self, n):
        H, dk, dv = self.cfg["n_kv_heads"], self.cfg["d_k"], self.cfg["d_v"]
        k = (self.rng.normal(size=(H, n, dk)) * self.sigma + self.mu).astype(np.float16)
        return k, self.rng.normal(size=(H, n, dv)).astype(np.float16)

    def prefill(self, b, L):
        k, v = self.tokens(L)
        self.gc.prefill_sequence(b, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda())
        self.oc[b] = self.oracle()
        self.oc[b].prefill(k[None], v[None])

    def chunk(self, T):
        """q, k_new, v_new of T tokens for every sequence (numpy fp16)."""
        B, Hq = self.cfg["batch"], self.cfg["n_q_heads"]
        kv = [self.tokens(T) for _ in range(B)]
        q = self.rng.normal(size=(B, Hq, T, self.cfg["d_k"])).astype(np.float16)
        return q, np.stack([x[0] for x in kv]), np.stack([x[1] for x in kv])

    def append_oracle(self, b, k, v):
        """k, v [Hkv][n][d]: n one-token appends to sequence b's oracle."""
        for i in range(k.shape[1]):
            self.oc[b].append(k[None, :, i], v[None, :, i])

    def check_state(self, where):
        for b, oc in enumerate(self.oc):
            if oc is not None:
                compare_state(self.gc, oc, b_rows=[b], where=f"{where} b={b}", seq=b)


def causal(T):
    return np.tril(np.ones((T, T), bool))


def reference(tw, b, q, k_new, v_new, sees):
    """fp64 outputs of sequence b's rows and the elementwise bound on an fp16 kernel's error.

    The bound, with u = 2^-11 (half a step of fp16), p_j the softmax weights and o the exact
    output: the output's own rounding u |o|; a weight and a value rounded to fp16 once each,
    2 u sum_j p_j |v_j|; keys (and the query side of a side code) rounded to fp16 once, which
    moves score j by at most d_j = u sum_c |q_c k_jc| / sqrt(d_k) and so the output by
    sum_j p_j d_j |v_j - o| to first order.  The kernel for few rows rounds the products q_c s_c
    of query and key scale instead: an error u |q_c s_c code| with s_c code = k_jc - z_c, z_c being
    the group's smallest key, so |k_jc| + max |k_.c| over the group takes the place of |k_jc|; and
    the weights' products with the value scale instead of weight and value, where likewise
    |s code| <= |v_j| + |z_j|, z_j the smallest value of the token's group.  The factor 1.05 covers the second order and the
    fp32 sums (relative 2^-24 a step over at most a few thousand steps)."""
    cfg = tw.cfg
    oc = tw.oc[b]
    n = q.shape[1]
    n_rep, dk = cfg["n_q_heads"] // cfg["n_kv_heads"], cfg["d_k"]
    if cfg.get("rot_keys"):
        o = tw.oracle()
        q, k_new = O.rotate_rows(q, o.sigma, o.cq), O.rotate_rows(k_new, o.sigma, o.ck)
    out = np.zeros(q.shape[:2] + (cfg["d_v"],))
    bound = np.zeros_like(out)
    for h in range(cfg["n_kv_heads"]):
        kk, vv = k_new[h].astype(np.float64), v_new[h].astype(np.float64)
        L = 0
        zh = None
        ka, va = np.abs(kk), np.abs(vv)
        if oc is not None:
            kh, vh = oc.decoded_kv(0, h)
            L = kh.shape[0]
            kk, vv = np.concatenate([kh, kk]), np.concatenate([vh, vv])
            Q, gk, gv = oc.Q, cfg["group_k"], cfg["group_v"]
            ka, va = np.abs(kk), np.abs(vv)
            if Q:
                ka[:Q] += np.repeat(np.abs(kh[:Q]).reshape(Q // gk, gk, -1).max(1), gk, axis=0)
                va[:Q] += np.repeat(np.abs(vh[:Q]).reshape(Q, -1, gv).max(2), gv, axis=1)
            if cfg.get("side_rank"):
                zh = oc.decoded_side(0, h)
        for r in range(n_rep):
            hq = h * n_rep + r
            qq = q[hq].astype(np.float64)
            s = qq @ kk.T
            mag = np.abs(qq) @ ka.T
            if zh is not None:
                qt = np.stack([O.side_query(oc.U[h], x) for x in qq])
                s[:, :L] += qt @ zh.T
                mag[:, :L] += 2 * np.abs(qt) @ np.abs(zh).T
            s /= math.sqrt(dk)
            s[:, L:][~sees[:n, :n]] = -np.inf
            seen = np.isfinite(s).any(1)
            p = np.exp(s - np.where(seen, s.max(1, initial=-np.inf), 0.0)[:, None])
            p /= np.maximum(p.sum(1, keepdims=True), 1e-300)
            o = p @ vv
            out[hq] = o
            delta = U16 * mag / math.sqrt(dk)
            spread = np.einsum("tj,tjc->tc", p * delta, np.abs(vv[None] - o[:, None]))
            bound[hq] = 1.05 * (U16 * np.abs(o) + 2 * U16 * (p @ va) + spread) + 2.0 ** -25
    return out, bound


def check_chunk(tw, T, counts=None, sees=None, splits=(0,), q_scale=1.0, kernels=KERNELS):
    q, k_new, v_new = tw.chunk(T)
    q = (q * np.float16(q_scale)).astype(np.float16)
    B = tw.cfg["batch"]
    n = [T] * B if counts is None else counts
    mask = None
    if sees is not None:
        words = np.zeros((B, T, -(-T // 32)), np.uint32)
        for b in range(B):
            for j in range(T):
                words[b, :, j // 32] |= sees[b][:, j].astype(np.uint32) << np.uint32(j % 32)
        mask = torch.from_numpy(words.view(np.int32)).cuda()
    # rows behind the valid ones must not be read: poison them
    kp, vp = k_new.copy(), v_new.copy()
    qp = q.copy()
    for b in range(B):
        kp[b, :, n[b]:], vp[b, :, n[b]:], qp[b, :, n[b]:] = np.nan, np.inf, np.nan
    args = [torch.from_numpy(x).cuda() for x in (qp, kp, vp)]
    refs = [reference(tw, b, q[b][:, :n[b]], k_new[b][:, :n[b]], v_new[b][:, :n[b]],
                      causal(T) if sees is None else sees[b]) for b in range(B)]
    for kern in kernels:
        tw.gc.set_kernel(kern)
        for ns in splits:
            out = torch.full(q.shape[:3] + (tw.cfg["d_v"],), 7.0, dtype=torch.float16, device="cuda")
            got = tw.gc.chunk_attention(*args, counts=counts, mask=mask, out=out, num_splits=ns)
            got = got.float().cpu().numpy().astype(np.float64)
            for b in range(B):
                ref, bound = refs[b]
                assert np.all(got[b, :, n[b]:] == 7.0), "a row behind the new tokens was written"
                if n[b] == 0:
                    continue
                bad = np.abs(got[b, :, :n[b]] - ref) > bound
                assert not bad.any(), (f"kernel {kern} splits {ns} b={b}: {bad.sum()} of {bad.size} outside the "
                                       f"bound, at {np.argwhere(bad)[:4].tolist()}, worst "
                                       f"{(np.abs(got[b, :, :n[b]] - ref) / bound).max():.2f} bounds")
    tw.gc.set_kernel(K.KVQ_KERNEL_AUTO)
    assert tw.gc.status() == 0


# ------------------------------------------------------------------ chunk attention ----
@pytest.mark.parametrize("T", [1, 2, 5, 31, 70])
def test_chunk_lengths(T):
    check_chunk(Twin(config(), [700, 129, 513], seed=T), T, splits=(0, 1, 3))


def test_chunk_of_a_prompt():
    check_chunk(Twin(config(batch=1, n_q_heads=4, n_kv_heads=1), [389], seed=3), 300, splits=(0, 2))


@pytest.mark.parametrize("lengths", [[1, 64, 127], [128, 191, 192], [193, 0, 5], [0, 0, 0]])
def test_chunk_over_short_and_empty_caches(lengths):
    check_chunk(Twin(config(), lengths, seed=sum(lengths)), 4, splits=(0, 1))


@pytest.mark.parametrize("kb,vb", [(8, 4), (2, 2), (4, 4), (8, 8), (2, 4), (4, 8), (16, 16)])
@pytest.mark.parametrize("T", [2, 3, 6, 20, 40])       # 8, 12, 24, 80 and 160 query rows of a kv head
def test_chunk_bit_widths(kb, vb, T):
    check_chunk(Twin(config(k_bits=kb, v_bits=vb), [600, 601, 333], seed=kb * 10 + vb), T,
                kernels=KERNELS if T == 6 else KERNELS[:1])


@pytest.mark.parametrize("dk,dv,kb", [(32, 128, 4), (64, 128, 4), (128, 64, 4), (256, 256, 4), (32, 32, 4), (32, 128, 2),
                                      (64, 128, 2), (32, 128, 8), (64, 128, 8)])
@pytest.mark.parametrize("T", [3, 5, 45])
def test_chunk_head_dims(dk, dv, kb, T):
    check_chunk(Twin(config(d_k=dk, d_v=dv, k_bits=kb, group_v=32, group_k=32), [400, 257, 90], seed=dk + dv), T)


@pytest.mark.parametrize("n_q,n_kv", [(2, 2), (4, 2), (16, 2), (3, 1)])
def test_chunk_query_groups(n_q, n_kv):
    check_chunk(Twin(config(n_q_heads=n_q, n_kv_heads=n_kv), [300, 450, 129], seed=n_q), 7)


@pytest.mark.parametrize("gk,gv,R,ret", [(16, 16, 0, 1), (32, 32, 64, 0), (128, 128, 5, 1), (64, 32, 300, 1),
                                         (32, 64, 1, 0)])
@pytest.mark.parametrize("T", [3, 8, 40])
def test_chunk_group_sizes_and_windows(gk, gv, R, ret, T):
    check_chunk(Twin(config(group_k=gk, group_v=gv, window=R, log_retain=ret), [777, 130, 33], seed=gk), T)


@pytest.mark.parametrize("extra", [
    dict(side_rank=4, side_bits=4), dict(side_rank=8, side_bits=4, rot_keys=1), dict(rot_keys=1), dict(paged=1),
    dict(paged=1, side_rank=4, side_bits=8, k_bits=2), VAR, dict(VAR, paged=1)])
@pytest.mark.parametrize("T", [1, 4, 7, 17, 45])
def test_chunk_cache_forms(extra, T):
    check_chunk(Twin(config(**extra), [640, 300, 127], seed=11), T, splits=(0, 2))


@pytest.mark.parametrize("extra", [
    VAR, dict(VAR, paged=1), dict(VAR, n_q_heads=2), dict(VAR, log_retain=0, window=0),
    dict(k_bits=0, v_bits=0, k_widths=[8] * 32 + [2] * 96, v_widths=[4] * 64 + [2] * 64),
    dict(k_bits=0, v_bits=0, group_v=32, k_widths=[4] * 64 + [2] * 64, v_widths=[4] * 64 + [2] * 64),
    dict(k_bits=0, v_bits=0, group_v=16, group_k=16, k_widths=[4] * 128, v_widths=[2] * 128)])
@pytest.mark.parametrize("T,counts", [(5, [5, 0, 2]), (17, [17, 16, 1]), (32, [32, 32, 32]), (3, [0, 0, 0])])
def test_chunk_width_maps(extra, T, counts):
    """The decode steps of a width map's chunk: both head groupings the decode kernel has, the maps
    built in and others, more tokens than are merged at a time, an empty cache."""
    lengths = [0, 640, 65] if T != 32 else [513] * 3
    check_chunk(Twin(config(**extra), lengths, seed=T), T, counts=counts, splits=(0, 1, 3),
                kernels=(K.KVQ_KERNEL_TENSOR,))


@pytest.mark.parametrize("extra", [VAR, dict(VAR, n_q_heads=4)])
def test_chunk_width_maps_by_size(extra):
    """The automatic choice on either side of its size rule, and a head grouping of no tensor kernel."""
    check_chunk(Twin(config(**extra, batch=1, max_context=5000), [4500], seed=5), 3)


@pytest.mark.parametrize("T,counts", [(5, [5, 0, 2]), (40, [1, 40, 33]), (3, [0, 0, 0])])
def test_chunk_counts_leave_the_other_rows_alone(T, counts):
    check_chunk(Twin(config(), [300, 500, 40], seed=T), T, counts=counts)


@pytest.mark.parametrize("T", [8, 37])
def test_chunk_masks(T):
    """Trees, arbitrary patterns, rows that see no new token, tokens that nobody sees."""
    tw = Twin(config(), [300, 0, 64], seed=T)
    rng = np.random.default_rng(T)
    tree = np.eye(T, dtype=bool)
    for j in range(1, T):
        tree[j] |= tree[rng.integers(max(0, j - 3), j)]
    anyhow = rng.random((T, T)) < 0.3
    anyhow[T // 2] = False                          # over an empty cache: a row of zeros
    check_chunk(tw, T, sees=[tree, anyhow, np.zeros((T, T), bool)], counts=[T, T, T - 1], splits=(0, 1))


def test_chunk_weighs_every_visible_token_once():
    """A query of zeros weighs all visible tokens alike, whatever the keys: the output is the
    mean of the values and the bound has no key term, so one token missing or counted twice
    (among fewer than about a thousand) shows."""
    check_chunk(Twin(config(), [640, 333, 130], seed=9), 9, q_scale=0.0, splits=(0, 1, 3))
    check_chunk(Twin(config(paged=1, group_k=16, group_v=16, window=7), [200, 0, 17], seed=8), 34, q_scale=0.0)
    check_chunk(Twin(config(batch=1, n_q_heads=4, n_kv_heads=1, window=64), [500], seed=8), 290, q_scale=0.0)


def test_chunk_scores_far_apart():
    """Queries 8 times as long: the running maximum moves often and most weights vanish."""
    check_chunk(Twin(config(), [640, 333, 130], seed=19), 9, q_scale=8.0, splits=(0, 1))


def test_chunk_of_one_is_the_next_decode():
    """One new token attended, then appended and decoded: the same attention (no group leaves
    the window here), within two outputs' roundings of each other and the fp16 path's bound."""
    tw = Twin(config(), [300, 300, 300], seed=2)
    q, k, v = [torch.from_numpy(x).cuda() for x in tw.chunk(1)]
    tw.gc.set_kernel(K.KVQ_KERNEL_GENERIC)
    a = tw.gc.chunk_attention(q, k, v)[:, :, 0].float()
    tw.gc.append_tokens(k, v)
    b = tw.gc.decode(q[:, :, 0].contiguous()).float()
    # two fp32 computations rounded to fp16 each: a step of the larger, plus fp32 noise
    assert torch.all((a - b).abs() <= 2 * U16 * torch.maximum(a.abs(), b.abs()) + 1e-5)


def test_chunk_and_append_far_into_a_large_cache():
    """Element offsets beyond 2^31: the last heads of an fp16 cache of 2.2 million slots."""
    need_gpu()
    tw = Twin(config(batch=1, n_q_heads=16, n_kv_heads=8, k_bits=16, v_bits=16, max_context=2200000), [0])
    k, v = tw.tokens(300)
    tw.gc.prefill_sequence(0, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda())
    small = O.OracleCache(dict(tw.cfg, max_context=400))
    small.prefill(k[None], v[None])
    tw.oc[0] = small
    for T in (2, 40, 80):
        check_chunk(tw, T, kernels=KERNELS[:1])
    _, kn, vn = tw.chunk(5)
    tw.gc.append_tokens(torch.from_numpy(kn).cuda(), torch.from_numpy(vn).cuda())
    tw.append_oracle(0, kn[0], vn[0])
    assert np.array_equal(tw.gc.view("win_k")[0, :, :305].cpu().numpy(), small.win_k[0, :, :305])
    assert np.array_equal(tw.gc.view("win_v")[0, :, :305].cpu().numpy(), small.win_v[0, :, :305])


def test_chunk_calls_on_two_streams_do_not_meet():
    """Two calls on one cache at once: each has its own workspace."""
    tw = Twin(config(), [900, 700, 800], seed=14)
    qa = [torch.from_numpy(x).cuda() for x in tw.chunk(3)]
    qb = [torch.from_numpy(x).cuda() for x in tw.chunk(30)]
    wa, wb = tw.gc.chunk_attention(*qa), tw.gc.chunk_attention(*qb)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(8):
        outs.append((tw.gc.chunk_attention(*qa, stream=s1), tw.gc.chunk_attention(*qb, stream=s2)))
    torch.cuda.synchronize()
    assert all(torch.equal(a, wa) and torch.equal(b, wb) for a, b in outs)


def test_chunk_large_values_and_keys():
    """Values up to a thousand and keys up to a hundred: no product of a weight and a scale leaves fp16."""
    tw = Twin(config(v_bits=2), [0, 0, 0], seed=15)
    for b, L in enumerate((400, 300, 200)):
        k, v = tw.tokens(L)
        k, v = (k * 10).astype(np.float16), (v * 300).astype(np.float16)
        tw.gc.prefill_sequence(b, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda())
        tw.oc[b] = tw.oracle()
        tw.oc[b].prefill(k[None], v[None])
    for T in (1, 4, 8, 20, 40):
        check_chunk(tw, T, kernels=KERNELS[:1])


def test_chunk_refusals():
    tw = Twin(config(), [300, 300, 300])
    q, k, v = [torch.from_numpy(x).cuda() for x in tw.chunk(4)]
    gc = tw.gc
    for bad in (dict(counts=[1, 2]), dict(counts=[5, 0, 0]), dict(counts=[-1, 0, 0]), dict(num_splits=-1),
                dict(mask=torch.zeros(3, 4, 2, dtype=torch.int32, device="cuda")),
                dict(mask=torch.zeros(3, 4, 1, dtype=torch.int64, device="cuda")),
                dict(mask=torch.zeros(3, 4, 1, dtype=torch.int32)),
                dict(out=torch.zeros(3, 8, 4, 64, dtype=torch.float16, device="cuda"))):
        with pytest.raises((ValueError, K.KVQError)):
            gc.chunk_attention(q, k, v, **bad)
    with pytest.raises(ValueError):
        gc.chunk_attention(q.float(), k, v)
    with pytest.raises(ValueError):
        gc.chunk_attention(q.transpose(1, 2), k, v)
    with pytest.raises(ValueError):
        gc.chunk_attention(q, k[:, :, :2].contiguous(), v)
    none = torch.zeros(3, 2, 0, 128, dtype=torch.float16, device="cuda")
    with pytest.raises(K.KVQError):
        gc.chunk_attention(torch.zeros(3, 8, 0, 128, dtype=torch.float16, device="cuda"), none, none)
    st = gc.workspace.data_ptr()
    args = (q.data_ptr(), k.data_ptr(), v.data_ptr(), 4, None, None, q.data_ptr())
    need = K.kvq_chunk_workspace_size(gc.handle, 4, 3)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    for a, code in ((args + (ws.data_ptr(), need - 1, 3, st, 0), K.KVQ_ERR_WORKSPACE),
                    (args + (ws.data_ptr() + 4, need, 3, st, 0), K.KVQ_ERR_ALIGN),
                    (args + (ws.data_ptr(), need, 3, None, 0), K.KVQ_ERR_INVALID_ARG),
                    (args + (None, need, 3, st, 0), K.KVQ_ERR_INVALID_ARG)):
        with pytest.raises(K.KVQError) as e:
            K.kvq_chunk_attention(gc.handle, *a)
        assert e.value.code == code


def test_chunk_captured_and_on_another_stream():
    tw = Twin(config(), [700, 300, 400], seed=4)
    q, k, v = [torch.from_numpy(x).cuda() for x in tw.chunk(5)]
    want = tw.gc.chunk_attention(q, k, v)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = tw.gc.chunk_attention(q, k, v, stream=side)
    side.synchronize()
    assert torch.equal(want, got)
    graphs, outs = [], []
    for _ in range(2):                        # two graphs of the same cache, replayed in turn
        out = torch.zeros_like(want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            tw.gc.chunk_attention(q, k, v, out=out)
        graphs.append(g)
        outs.append(out)
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


# ------------------------------------------------------------------ multi-token append ----
def check_append(tw, T, counts, index=None, where=""):
    _, k, v = tw.chunk(T)
    B = tw.cfg["batch"]
    n = [T] * B if counts is None else counts
    kp, vp = k.copy(), v.copy()
    idx = None
    if index is not None:
        idx = torch.from_numpy(np.asarray(index, np.int32)).cuda()
    else:
        for b in range(B):
            kp[b, :, n[b]:], vp[b, :, n[b]:] = np.nan, np.nan
    tw.gc.append_tokens(torch.from_numpy(kp).cuda(), torch.from_numpy(vp).cuda(), counts=counts, index=idx)
    for b in range(B):
        if n[b]:
            rows = list(range(n[b])) if index is None else [int(i) for i in index[b][:n[b]]]
            tw.append_oracle(b, k[b][:, rows], v[b][:, rows])
    tw.check_state(where)


@pytest.mark.parametrize("extra", [
    dict(), dict(log_retain=0, group_k=16, group_v=16, window=0), dict(group_k=32, group_v=32, window=5, k_bits=8, v_bits=4),
    dict(k_bits=16, v_bits=16), dict(rot_keys=1), dict(side_rank=4, side_bits=4), dict(side_rank=8, side_bits=4, rot_keys=1),
    dict(paged=1), dict(paged=1, side_rank=4, side_bits=8, k_bits=2), VAR, dict(VAR, paged=1), dict(d_k=32, k_bits=2),
    dict(d_k=256, d_v=256, group_k=128, group_v=8, k_bits=8, v_bits=8), dict(d_k=32, d_v=64, group_v=32)])
def test_append_tokens_is_that_many_appends(extra):
    tw = Twin(config(**extra), [300, 128, 1], seed=21)
    for T, counts in ((1, None), (4, [4, 0, 2]), (3, [0, 0, 0]), (150, [150, 7, 149]), (64, [1, 64, 63])):
        check_append(tw, T, counts, where=f"T={T}")
    # one-token appends go on from there
    _, k, v = tw.chunk(1)
    tw.gc.append(torch.from_numpy(k[:, :, 0]).cuda(), torch.from_numpy(v[:, :, 0]).cuda())
    for b in range(3):
        tw.append_oracle(b, k[b], v[b])
    tw.check_state("append after append_tokens")


def test_append_tokens_by_index():
    tw = Twin(config(), [190, 191, 130], seed=5)
    check_append(tw, 6, [3, 6, 4], index=[[5, 0, 2, -1, 99, 7], [1, 1, 1, 1, 1, 1], [3, 2, 1, 0, 0, 0]])
    check_append(tw, 70, [70, 1, 66], index=[list(range(69, -1, -1)), [69] * 70, [i // 2 for i in range(70)]])


def test_append_tokens_uniform_lengths():
    tw = Twin(config(), [190, 190, 190], seed=6)
    for T in (1, 2, 200):
        check_append(tw, T, None, where=f"uniform T={T}")


def test_append_tokens_refusals():
    tw = Twin(config(max_context=320), [300, 310, 0])
    _, k, v = [torch.from_numpy(x).cuda() for x in tw.chunk(16)]
    before = [tw.gc.seq_state(b) for b in range(3)]
    for counts, code in (([16, 11, 0], K.KVQ_ERR_CAPACITY), ([1, 1, 1], K.KVQ_ERR_STATE), ([17, 0, 0], K.KVQ_ERR_INVALID_ARG),
                         ([0, -1, 0], K.KVQ_ERR_INVALID_ARG)):
        with pytest.raises(K.KVQError) as e:
            tw.gc.append_tokens(k, v, counts=counts)
        assert e.value.code == code
    with pytest.raises(ValueError):
        tw.gc.append_tokens(k, v, counts=[1, 0, 0], index=torch.zeros(3, 15, dtype=torch.int32, device="cuda"))
    assert [tw.gc.seq_state(b) for b in range(3)] == before
    tw.check_state("after refusals")
    check_append(tw, 16, [16, 10, 0])


def test_append_tokens_with_an_exhausted_pool_changes_nothing():
    tw = Twin(config(paged=1, n_pages=6), [320, 256, 192], seed=3)      # 3 + 2 + 1 pages
    assert tw.gc.free_pages() == 0
    _, k, v = [torch.from_numpy(x).cuda() for x in tw.chunk(64)]
    with pytest.raises(K.KVQError) as e:
        tw.gc.append_tokens(k, v, counts=[64, 0, 0])
    assert e.value.code == K.KVQ_ERR_CAPACITY
    tw.check_state("exhausted")
    check_append(tw, 64, [63, 63, 63])


# ------------------------------------------------------------------ forks ----
@pytest.mark.parametrize("extra", [dict(), dict(paged=1), dict(paged=1, side_rank=4, side_bits=4, rot_keys=1),
                                   dict(side_rank=8, side_bits=4), dict(k_bits=16, v_bits=16), VAR, dict(VAR, paged=1),
                                   dict(d_k=32, d_v=32, group_v=32, window=0, group_k=16, k_bits=2)])
def test_fork_copies_and_then_diverges(extra):
    tw = Twin(config(batch=5, **extra), [700, 131, 200, 0, 0], seed=7)
    gc = tw.gc
    pages = gc.free_pages()
    gc.fork([0, 0, 1], [2, 3, 4])          # two branches of 0; slot 2 gives up what it held
    import copy
    for s, d in ((0, 2), (0, 3), (1, 4)):
        tw.oc[d] = copy.deepcopy(tw.oc[s])
    if extra.get("paged"):
        gk = tw.cfg["group_k"]
        assert gc.free_pages() == pages + O.quantized_prefix(200, tw.cfg["window"], gk, 4) // gk
    tw.check_state("fork")
    for T, counts in ((40, [40, 3, 17, 0, 40]), (90, [5, 90, 64, 80, 1])):
        check_append(tw, T, counts, where="diverging")
    check_chunk(tw, 3)
    gc.release(0)                           # the parent ends; its branches keep their tokens
    tw.oc[0] = None
    tw.prefill(1, 260)                      # and slot 1 starts over
    tw.check_state("parent released")
    check_chunk(tw, 2, counts=[0, 2, 2, 2, 2])
    assert gc.status() == 0


def test_fork_shares_pages_until_the_last_holder_leaves():
    tw = Twin(config(batch=3, paged=1, n_pages=12), [512, 0, 0], seed=8)       # 6 pages
    gc = tw.gc
    gc.fork([0, 0], [1, 2])
    assert gc.free_pages() == 6
    gc.release(0)
    gc.release(0)                           # releasing an empty sequence frees nothing more
    gc.release(1)
    assert gc.free_pages() == 6
    gc.release(2)
    assert gc.free_pages() == 12
    # a whole-batch prefill takes shared pages back as well
    tw.prefill(0, 512)
    gc.fork(0, 1)
    k, v = zip(*[tw.tokens(384) for _ in range(3)])                            # 3 x 4 pages
    gc.prefill(torch.from_numpy(np.stack(k)).cuda(), torch.from_numpy(np.stack(v)).cuda())
    assert gc.free_pages() == 0
    # and a single prefill counts only the pages that it would free
    gc.fork(0, 1)
    assert gc.free_pages() == 4
    with pytest.raises(K.KVQError) as e:
        tw.prefill(1, 128 + 5 * 64)
    assert e.value.code == K.KVQ_ERR_CAPACITY


def test_fork_refusals_change_nothing():
    tw = Twin(config(batch=4, paged=1), [300, 200, 0, 129], seed=1)
    pages = tw.gc.free_pages()
    for src, dst, code in (([0, 1], [2, 2], K.KVQ_ERR_INVALID_ARG), ([0, 3], [3, 2], K.KVQ_ERR_INVALID_ARG),
                           ([0], [0], K.KVQ_ERR_INVALID_ARG), ([4], [2], K.KVQ_ERR_INVALID_ARG),
                           ([0], [-1], K.KVQ_ERR_INVALID_ARG), ([0, 2], [3, 1], K.KVQ_ERR_STATE)):
        with pytest.raises(K.KVQError) as e:
            tw.gc.fork(src, dst)
        assert e.value.code == code
    with pytest.raises(ValueError):
        tw.gc.fork([0], [1, 2])
    tw.gc.fork([], [])
    assert tw.gc.free_pages() == pages
    tw.check_state("refused forks")


def test_fork_many_at_once():
    """More pairs than one launch takes."""
    need_gpu()
    cfg = config(batch=601, n_q_heads=1, n_kv_heads=1, d_k=32, d_v=32, group_k=16, group_v=16, window=3,
                 max_context=64, log_retain=0)
    tw = Twin(cfg, [50] + [0] * 600, seed=3)
    tw.gc.fork([0] * 600, list(range(1, 601)))
    for name in ("kcode", "ksz", "vcode", "vsz", "win_k", "win_v"):
        t = tw.gc.view(name)
        assert torch.equal(t, t[:1].expand_as(t)), name
    assert tw.gc.seq_state(600) == tw.gc.seq_state(0)


# ------------------------------------------------------------------ compaction ----
@pytest.mark.parametrize("extra", [dict(), dict(side_rank=4, side_bits=4), dict(k_bits=8, v_bits=8, group_k=16, group_v=16), VAR])
def test_compaction_moves_pages_and_nothing_else(extra):
    tw = Twin(config(batch=6, paged=1, **extra), [700, 300, 129, 650, 500, 0], seed=13)
    gc, gk = tw.gc, tw.cfg["group_k"]
    gc.fork(3, 5)                           # a shared page moves once
    tw.oc[5] = __import__("copy").deepcopy(tw.oc[3])
    for b in (0, 2):
        gc.release(b)
        tw.oc[b] = None
    tw.prefill(2, 400)
    n = tw.cfg["n_pages"]
    for end in ("low", "low", "high", "low", "high"):
        free = gc.free_pages()
        used = gc.compact(end)
        assert used == n - free and gc.free_pages() == free
        table = gc.view("block_table").cpu()
        held = {int(p) for b in range(6) if tw.oc[b] is not None for p in table[b, :tw.oc[b].Q // gk]}
        assert held == set(range(used) if end == "low" else range(n - used, n))
        tw.check_state(f"compact {end}")
        check_chunk(tw, 2, counts=[0, 2, 1, 2, 2, 2], kernels=(K.KVQ_KERNEL_AUTO,))
        check_append(tw, 70, [0, 70, 3, 70, 1, 64], where="append after compaction")


def test_compaction_of_large_and_empty_pools():
    need_gpu()
    cfg = config(batch=4, n_q_heads=1, n_kv_heads=1, d_k=32, d_v=32, group_k=16, group_v=16, window=0,
                 max_context=40000, log_retain=0, paged=1, n_pages=11000)
    tw = Twin(cfg, [0] * 4)
    assert tw.gc.compact("high") == 0 and tw.gc.free_pages() == 11000
    gen = torch.Generator(device="cuda").manual_seed(1)
    for b in range(4):                      # 2500 pages each
        kv = torch.randn((2, 1, 40000, 32), generator=gen, device="cuda").half()
        tw.gc.prefill_sequence(b, kv[0].contiguous(), kv[1].contiguous())
    before = {(n, b): tw.gc.sequence_view(n, b) for n in ("kcode", "ksz", "vcode", "vsz") for b in (1, 3)}
    tw.gc.release(0)
    tw.gc.release(2)
    for end in ("high", "low"):             # more moves than one launch takes
        assert tw.gc.compact(end) == 5000
        for (n, b), t in before.items():
            assert torch.equal(tw.gc.sequence_view(n, b), t), (end, n, b)


def test_compaction_refusals():
    tw = Twin(config(), [300, 200, 129])
    with pytest.raises(K.KVQError) as e:
        tw.gc.compact()
    assert e.value.code == K.KVQ_ERR_UNSUPPORTED
    with pytest.raises(ValueError):
        tw.gc.compact("middle")
    with pytest.raises(K.KVQError) as e:
        K.kvq_compact_pages(tw.gc.handle, 2, 0)
    assert e.value.code == K.KVQ_ERR_INVALID_ARG


# ------------------------------------------------------------------ all of it together ----
@pytest.mark.parametrize("extra", [dict(paged=1), dict()])
def test_speculative_serving_loop(extra):
    """Branches, draft trees, accepted paths and a compacted pool, step after step: the caches
    stay those of plain one-token appends."""
    import copy
    tw = Twin(config(batch=4, **extra), [500, 260, 0, 0], seed=31)
    gc = tw.gc
    gc.fork([0, 1], [2, 3])
    tw.oc[2], tw.oc[3] = copy.deepcopy(tw.oc[0]), copy.deepcopy(tw.oc[1])
    rng = np.random.default_rng(0)
    T = 7
    for step in range(12):
        tree = [np.eye(T, dtype=bool) for _ in range(4)]
        paths = []
        for t in tree:
            parent = [-1] + [int(rng.integers(max(0, j - 3), j)) for j in range(1, T)]
            for j in range(1, T):
                t[j] |= t[parent[j]]
            leaf = int(rng.integers(0, T))
            paths.append([j for j in range(T) if t[leaf, j]])
        if step % 4 == 0:
            check_chunk(tw, T, sees=tree)
        check_append(tw, T, [len(p) for p in paths], index=[p + [0] * (T - len(p)) for p in paths], where=f"step {step}")
        if step == 5:
            gc.release(1)
            tw.oc[1] = None
            gc.fork(0, 1)
            tw.oc[1] = copy.deepcopy(tw.oc[0])
            if extra.get("paged"):
                gc.compact("low")
    q = rng.normal(size=(4, 8, 128)).astype(np.float16)
    out = gc.decode(torch.from_numpy(q).cuda()).float().cpu().numpy()
    for b in range(4):
        assert O.max_rel_error(out[b:b + 1], tw.oc[b].decode(q[b:b + 1])) <= 2e-3
