"""Vocabulary operators without a GPU: the oracle's formulas against brute
force and against differences, and every refusal that the header documents,
reported on the host before any device work."""
import numpy as np
import os
import pytest

import lm_head_gumbel_amd as fs
from oracle import vocab as OV

built = pytest.mark.skipif(not os.path.exists(fs.LIB_PATH),
                           reason="libfs.so not built (python -m lm_head_gumbel_amd.build)")
BAD, UNSUP = fs.FS_ERR_INVALID_ARG, fs.FS_ERR_UNSUPPORTED


def test_oracle_dequantises_by_hand():
    q = np.array([[0x21, 0xF0]], np.uint8)                       # 1, 2, 0, 15
    assert np.array_equal(OV.unpack_w4(q), [[1, 2, 0, 15]])
    assert np.array_equal(OV.dequantise(q, [[0.5, 2.0]], None, 2), [[-3.5, -3.0, -16.0, 14.0]])
    assert np.array_equal(OV.dequantise(q, [[0.5, 2.0]], [[1, 200]], 2), [[0, 0.5, -400, -370]])


def test_oracle_logprobs_by_hand():
    l = OV.clean_logits(np.array([[0.0, np.log(3.0), 0.0, np.nan], [1, 1, 1, 1]]), None,
                        np.array([[0xF], [0xB]], np.uint32))
    r = OV.logprobs(l, np.ones(2), [2, 3], 4)
    assert np.allclose(np.exp(r["logprob"]), [0.2, 1 / 3])
    assert r["rank"].tolist() == [3, 3]
    assert r["top_idx"].tolist() == [[1, 0, 2, -1], [0, 1, 3, -1]]
    assert np.allclose(r["lse"], [np.log(5), 1 + np.log(3)])
    assert np.allclose(r["entropy"], [-(0.6 * np.log(0.6) + 0.4 * np.log(0.2)), np.log(3)])


def loss(l, T, token, top_idx, g):
    r = OV.logprobs(l, T, token, 0)
    total = (g["lp"] * r["logprob"]).sum() + (g["lse"] * r["lse"]).sum() + (g["ent"] * r["entropy"]).sum()
    for b in range(l.shape[0]):
        for j in range(top_idx.shape[1]):
            if top_idx[b, j] >= 0:
                total += g["top"][b, j] * (l[b, top_idx[b, j]] / T[b] - r["lse"][b])
    return total


def test_oracle_gradient_against_differences():
    rng = np.random.default_rng(3)
    B, V = 3, 9
    l = OV.clean_logits(rng.normal(size=(B, V)), 8, rng.integers(0, 2 ** 9, (B, 1), dtype=np.uint32) | 3)
    T = np.array([0.7, 1.0, 1.6])
    token = np.array([1, 0, 1])
    r = OV.logprobs(l, T, token, 3)
    g = dict(lp=rng.normal(size=B), lse=rng.normal(size=B), ent=rng.normal(size=B), top=rng.normal(size=(B, 3)))
    got, _ = OV.logprobs_grad(l, T, token, r["top_idx"], r["lse"], r["entropy"], g["lp"], g["lse"], g["ent"], g["top"])
    for b in range(B):
        for i in range(V):
            if l[b, i] == -np.inf:
                assert got[b, i] == 0
                continue
            h = 1e-5
            up, dn = l.copy(), l.copy()
            up[b, i] += h
            dn[b, i] -= h
            d = (loss(up, T, token, r["top_idx"], g) - loss(dn, T, token, r["top_idx"], g)) / (2 * h)
            # central difference: h^2 / 6 of the third derivative, and rounding 1e-16 / h
            assert abs(d - got[b, i]) < 1e-8


def test_oracle_embed_by_hand():
    W = np.arange(6.0).reshape(3, 2)
    assert np.array_equal(OV.embed([18, 16, 15, -1], W, 2.0, 16), [[8, 10], [0, 2], [0, 0], [0, 0]])
    dW, mag = OV.embed_grad([1, -1, 1, 0, 3], np.array([[1.0, -1], [9, 9], [2, 3], [4, 5], [9, 9]]), 2.0, 3)
    assert np.array_equal(dW, [[8, 10], [6, 4], [0, 0]])
    assert np.array_equal(mag, [[8, 10], [6, 8], [0, 0]])


def quant(q=16, scale=16, zero=None, group=32, dt=fs.FS_F32):
    return fs.quant(q, scale, zero, group, dt)


@built
def test_quant_refusals():
    p = fs.params(2, 64, 128)
    call = fs.fs_logits_quant
    assert fs.lib().fs_logits_quant(None, 16, None, 16, None) == BAD
    assert call(p, 16, None, 16) == BAD
    assert call(p, 16, quant(dt=3), 16) == BAD
    assert call(p, 16, quant(dt=-1), 16) == BAD
    assert call(p, 16, quant(group=0), 16) == BAD
    assert call(p, 16, quant(group=-32), 16) == BAD
    assert call(p, 16, quant(), None) == BAD
    assert call(p, None, quant(), 16) == BAD
    assert call(p, 16, quant(q=None), 16) == BAD
    assert call(p, 16, quant(scale=None), 16) == BAD
    assert call(fs.params(2, 64, 128, flags=2), 16, quant(), 16) == BAD
    for group in (1, 16, 33, 96, 192, 320):
        assert call(fs.params(2, 9600, 128), 16, quant(group=group), 16) == UNSUP, group
    assert call(p, 16, quant(group=128), 16) == UNSUP              # does not divide d
    assert call(fs.params(2, 72, 128), 16, quant(), 16) == UNSUP
    assert call(p, 24, quant(), 16) == UNSUP                       # alignment
    assert call(p, 16, quant(q=8), 16) == UNSUP
    assert call(p, 16, quant(scale=18), 16) == UNSUP
    assert call(p, 16, quant(scale=17, dt=fs.FS_BF16), 16) == UNSUP
    assert call(fs.params(0, 64, 128), None, quant(None, None), None) == fs.FS_OK
    assert call(fs.params(2, 64, 0), None, quant(None, None), None) == fs.FS_OK


@built
def test_quant_row_limit():
    # ids of the last pass have to fit an int
    over = fs.params(1, 128, 2 ** 31 - 2 ** 20)
    assert fs.fs_logits_quant(over, 16, quant(), 16) == UNSUP
    assert fs.fs_logits_quant(over, 16, quant(group=96), None) == BAD


def lp(p, logits=16, token=16, n_top=0, logprob=16, idx=None, val=None, dtype=fs.FS_F32, ld=None, **kw):
    return fs.fs_logprobs(p, logits, None, None, token, n_top, logprob, None, None, None, idx, val, 256, 1 << 30,
                          dtype=dtype, ld=ld, **kw)


@built
def test_logprobs_refusals():
    p = fs.params(2, 0, 128)
    assert lp(fs.params(-1, 0, 128)) == BAD
    assert lp(p, dtype=3) == BAD
    assert lp(p, dtype=-1) == BAD
    assert lp(p, ld=127) == BAD
    assert lp(p, ld=-128) == BAD
    assert lp(p, logits=None) == BAD
    assert lp(p, token=None) == BAD
    assert lp(p, n_top=-1) == BAD
    assert lp(p, n_top=65, idx=16, val=16) == UNSUP
    assert lp(p, n_top=3, idx=16) == BAD
    assert lp(p, n_top=3, val=16) == BAD
    assert lp(p, logits=18) == UNSUP
    assert lp(p, logits=17, dtype=fs.FS_F16) == UNSUP
    assert lp(fs.params(2, 0, 128, v_offset=8)) == UNSUP
    assert lp(fs.params(0, 0, 128), None, None, logprob=None) == fs.FS_OK
    assert fs.fs_workspace_bytes(p, fs.FS_VARIANT_LOGPROBS, -1) == 0
    assert fs.fs_workspace_bytes(p, fs.FS_VARIANT_LOGPROBS, 65) == 0


def lpg(p, logits=16, token=16, n_top=0, top_idx=None, lse=16, entropy=16, g_lp=16, g_ent=16, g_top=None, grad=32,
        dtype=fs.FS_F32, ld=None, ld_grad=None):
    return fs.fs_logprobs_grad(p, logits, None, None, token, n_top, top_idx, lse, entropy, g_lp, None, g_ent, g_top, grad,
                               dtype=dtype, ld=ld, ld_grad=ld_grad)


@built
def test_logprobs_grad_refusals():
    p = fs.params(2, 0, 128)
    assert lpg(p, dtype=5) == BAD
    assert lpg(p, ld=100) == BAD
    assert lpg(p, ld_grad=100) == BAD
    assert lpg(p, logits=None) == BAD
    assert lpg(p, grad=None) == BAD
    assert lpg(p, lse=None) == BAD
    assert lpg(p, token=None) == BAD
    assert lpg(p, entropy=None) == BAD
    assert lpg(p, n_top=2, g_top=16) == BAD
    assert lpg(p, n_top=-2) == BAD
    assert lpg(p, n_top=65) == UNSUP
    assert lpg(p, grad=16, ld_grad=256) == BAD                     # in place: the same rows
    assert lpg(p, grad=34) == UNSUP
    assert lpg(fs.params(0, 0, 128), None, grad=None) == fs.FS_OK
    assert lpg(fs.params(2, 0, 0), None, grad=None) == fs.FS_OK


@built
def test_embed_refusals():
    p = fs.params(2, 33, 128)
    call = fs.fs_embed
    assert call(p, 16, 16, 1.0, 16, dtype=4) == BAD
    assert call(p, None, 16, 1.0, 16, dtype=0) == BAD
    assert call(p, 16, None, 1.0, 16, dtype=0) == BAD
    assert call(p, 16, 16, 1.0, None, dtype=0) == BAD
    assert call(p, 16, 18, 1.0, 16, dtype=0) == UNSUP
    assert call(p, 16, 16, 1.0, 17, dtype=1) == UNSUP
    assert call(fs.params(2, -1, 128), 16, 16, 1.0, 16, dtype=0) == BAD
    assert call(fs.params(0, 33, 128), None, None, 1.0, None, dtype=0) == fs.FS_OK
    assert call(fs.params(2, 0, 128), None, None, 1.0, None, dtype=0) == fs.FS_OK
    grad = lambda p, ids=16, g=16, acc=0, dW=16, dt=0, do=0: fs.fs_embed_grad(  # noqa: E731
        p, ids, g, 1.0, acc, dW, 256, 1 << 30, dtype=dt, dw_dtype=do)
    assert grad(p, dt=3) == BAD
    assert grad(p, do=3) == BAD
    assert grad(p, dt=fs.FS_BF16, do=fs.FS_F16) == UNSUP
    assert grad(p, dt=fs.FS_F32, do=fs.FS_BF16) == UNSUP
    assert grad(p, ids=None) == BAD
    assert grad(p, g=None) == BAD
    assert grad(p, dW=None) == BAD
    assert grad(p, g=18) == UNSUP
    assert grad(p, dW=18) == UNSUP
    assert grad(fs.params(0, 33, 128), None, None, 1) == fs.FS_OK
    assert grad(fs.params(2, 0, 128), None, None, dW=None) == fs.FS_OK
    assert grad(fs.params(2, 33, 0), None, None, dW=None) == fs.FS_OK


@built
def test_tensors_must_fit_the_call():
    torch = pytest.importorskip("torch")
    z = torch.zeros
    p = fs.params(2, 8, 4)
    out = z(2)
    args = dict(ws=z(8), ws_bytes=1 << 30)
    assert fs.fs_logprobs(p, z(2, 8)[:, ::2], None, None, z(2, dtype=torch.int32), 0, out, **args) == BAD
    assert fs.fs_logprobs(p, z(3, 4), None, None, z(2, dtype=torch.int32), 0, out, **args) == BAD
    assert fs.fs_logprobs(p, z(2, 4, dtype=torch.float64), None, None, z(2, dtype=torch.int32), 0, out, **args) == BAD
    assert fs.fs_logprobs(p, z(2, 4), None, None, z(4, dtype=torch.int32)[::2], 0, out, **args) == BAD
    ids = z(2, dtype=torch.int32)
    assert fs.fs_embed(p, ids, z(8, 4).T, 1.0, z(2, 8)) == BAD
    assert fs.fs_embed(p, ids, z(4, 8), 1.0, z(2, 8, dtype=torch.float16)) == BAD
    assert fs.fs_embed_grad(p, ids, z(8, 2).T, 1.0, 0, z(4, 8), z(8), 1 << 30) == BAD
    assert fs.fs_logits_quant(p, z(8, 2).T, quant(), z(2, 4)) == BAD
    with pytest.raises(ValueError):
        fs.quant(z(4, 4, dtype=torch.uint8).T, z(4, 1), None, 8)
