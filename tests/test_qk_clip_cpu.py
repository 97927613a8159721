"""QK-Clip: argument checks. Nothing is launched: every call here is refused before it looks for a device."""
import math

import pytest
import torch

import adamw_hybrid_optimizer_muon_b200 as ma

Q, K, OFF, OUT, WQ, WK = (0x6000_0000_0000 + k * (1 << 36) for k in range(6))  # made up, never followed


def top(seqs=2, len=100, total=0, heads=4, kv=2, dim=64, q=Q, q_seq=25600, q_tok=256, q_head=64, k=K, k_seq=12800,
        k_tok=128, k_head=64, offsets=None, scale=0.125, causal=1, absolute=0, accumulate=0, out=OUT):
    return ma.lib().ma_qk_max_logit(seqs, len, total, heads, kv, dim, q, q_seq, q_tok, q_head, k, k_seq, k_tok, k_head,
                                    offsets, scale, causal, absolute, accumulate, out, None)


def clip(heads=4, kv=2, q_rows=64, k_rows=64, cols=256, wq=WQ, wk=WK, top=OUT, tau=100.0, alpha=0.5):
    return ma.lib().ma_qk_clip(heads, kv, q_rows, k_rows, cols, wq, wk, top, tau, alpha, None)


@pytest.mark.parametrize("kw,code", [
    (dict(seqs=-1), ma.MA_ERR_SHAPE), (dict(len=-1), ma.MA_ERR_SHAPE), (dict(total=-1), ma.MA_ERR_SHAPE),
    (dict(heads=0), ma.MA_ERR_SHAPE), (dict(kv=0), ma.MA_ERR_SHAPE), (dict(kv=3), ma.MA_ERR_SHAPE),
    (dict(dim=0), ma.MA_ERR_SHAPE), (dict(dim=264), ma.MA_ERR_UNSUPPORTED), (dict(dim=60), ma.MA_ERR_ALIGN),
    (dict(len=1 << 31), ma.MA_ERR_UNSUPPORTED), (dict(seqs=1 << 31), ma.MA_ERR_UNSUPPORTED),
    (dict(heads=1 << 17, kv=1 << 17), ma.MA_ERR_UNSUPPORTED),
    (dict(scale=0.0), ma.MA_ERR_ARG), (dict(scale=-1.0), ma.MA_ERR_ARG), (dict(scale=math.nan), ma.MA_ERR_ARG),
    (dict(scale=math.inf), ma.MA_ERR_ARG), (dict(causal=2), ma.MA_ERR_ARG), (dict(absolute=3), ma.MA_ERR_ARG),
    (dict(accumulate=-1), ma.MA_ERR_ARG), (dict(out=None), ma.MA_ERR_NULL), (dict(out=OUT + 2), ma.MA_ERR_ALIGN),
    (dict(q=None), ma.MA_ERR_NULL), (dict(k=None), ma.MA_ERR_NULL), (dict(q=Q + 8), ma.MA_ERR_ALIGN),
    (dict(k=K + 2), ma.MA_ERR_ALIGN), (dict(q_tok=250), ma.MA_ERR_ALIGN), (dict(q_tok=32), ma.MA_ERR_SHAPE),
    (dict(k_head=0), ma.MA_ERR_SHAPE), (dict(k_seq=-8), ma.MA_ERR_SHAPE), (dict(q_seq=1 << 38), ma.MA_ERR_UNSUPPORTED),
    (dict(offsets=OFF + 2, total=100), ma.MA_ERR_ALIGN),
    (dict(len=1 << 30, heads=1 << 11, kv=1 << 11), ma.MA_ERR_UNSUPPORTED)])
def test_max_logit_refuses(kw, code):
    assert top(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(heads=0), ma.MA_ERR_SHAPE), (dict(kv=3), ma.MA_ERR_SHAPE), (dict(q_rows=-1), ma.MA_ERR_SHAPE),
    (dict(cols=-1), ma.MA_ERR_SHAPE), (dict(heads=2048, kv=1), ma.MA_ERR_UNSUPPORTED),
    (dict(cols=(1 << 30) + 1), ma.MA_ERR_UNSUPPORTED),
    (dict(q_rows=1 << 30, cols=1 << 30), ma.MA_ERR_UNSUPPORTED), (dict(k_rows=1 << 30, cols=1 << 30), ma.MA_ERR_UNSUPPORTED),
    (dict(tau=0.0), ma.MA_ERR_ARG), (dict(tau=math.nan), ma.MA_ERR_ARG),
    (dict(tau=math.inf), ma.MA_ERR_ARG), (dict(alpha=-0.1), ma.MA_ERR_ARG), (dict(alpha=1.1), ma.MA_ERR_ARG),
    (dict(alpha=math.nan), ma.MA_ERR_ARG), (dict(top=None), ma.MA_ERR_NULL), (dict(wq=None), ma.MA_ERR_NULL),
    (dict(wk=None), ma.MA_ERR_NULL), (dict(wq=WQ + 2), ma.MA_ERR_ALIGN), (dict(top=OUT + 1), ma.MA_ERR_ALIGN),
    (dict(wk=WQ + 4), ma.MA_ERR_ARG), (dict(top=WQ + 8), ma.MA_ERR_ARG), (dict(top=WK), ma.MA_ERR_ARG)])
def test_clip_refuses(kw, code):
    assert clip(**kw) == code


def test_host_tensors_are_refused():
    q = torch.zeros((1, 4, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ma.MAError) as e:
        ma.qk_max_logit(q, q)
    assert e.value.code == ma.MA_ERR_ARG
    w = torch.zeros((128, 64))
    with pytest.raises(ma.MAError) as e:
        ma.qk_clip(w, w.clone(), torch.zeros(2))
    assert e.value.code == ma.MA_ERR_ARG
