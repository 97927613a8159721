"""The largest logits are not written into what they are made of. Nothing is launched: the addresses are made up."""
import pytest

import adamw_hybrid_optimizer_muon_b200 as ma

Q, K, OFF, OUT = (0x6000_0000_0000 + k * (1 << 36) for k in range(4))
SEQS, LEN, HEADS, KV, DIM = 2, 100, 4, 2, 64
NQ, NK = SEQS * LEN * HEADS * DIM * 2, SEQS * LEN * KV * DIM * 2  # bytes


def top(out, offsets=None, q=Q, k=K):
    return ma.lib().ma_qk_max_logit(SEQS, LEN, SEQS * LEN if offsets else 0, HEADS, KV, DIM, q, LEN * HEADS * DIM,
                                    HEADS * DIM, DIM, k, LEN * KV * DIM, KV * DIM, DIM, offsets, 0.125, 1, 0, 0, out, None)


@pytest.mark.parametrize("offsets", [None, OFF])
@pytest.mark.parametrize("out", [Q, Q + 1024, Q + NQ - 4, Q - 12, K, K + NK - 4, K - 4])
def test_into_queries_or_keys(out, offsets):
    assert top(out, offsets) == ma.MA_ERR_ARG


@pytest.mark.parametrize("out", [OFF, OFF + 4 * SEQS, OFF - 12])
def test_into_the_offsets(out):
    assert top(out, OFF) == ma.MA_ERR_ARG


def test_queries_that_are_the_keys_are_one_input():
    # both are read: what is refused here comes after this check
    assert ma.lib().ma_qk_max_logit(1, 1 << 30, 0, 2048, 2048, DIM, Q, 0, 2048 * DIM, DIM, Q, 0, 2048 * DIM, DIM, None,
                                    0.125, 1, 0, 0, OUT, None) == ma.MA_ERR_UNSUPPORTED
