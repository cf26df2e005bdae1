"""What the serving calls' Python side refuses or keeps by itself; no GPU."""
from __future__ import annotations

import pytest
import torch

import io_aware_attention_fwd_gb300 as attn
from io_aware_attention_fwd_gb300 import api, build_ext

FAKE = 0x10000  # aligned, non-null, never dereferenced on these paths


@pytest.fixture(scope="module", autouse=True)
def built():
    build_ext.build()


BIG = [(1 << 32) + 10, -(1 << 32) + 10, 1 << 31]


def cache(**kw):
    args = dict(k_codes=FAKE, k_meta=FAKE, v_codes=FAKE, v_meta=FAKE, weight=FAKE, pos=FAKE, length=FAKE, B=3, H_kv=2,
                capacity=100, D=64)
    args.update(kw)
    return attn.attn_cache4_t(*args.values())


@pytest.mark.parametrize("big", BIG)
def test_numbers_beyond_an_int_are_refused(big):
    """None of them is taken as its low 32 bits (10), which every call here would accept."""
    c, invalid = cache(), attn.ATTN_ERR_INVALID_ARG
    ws = 1 << 40
    for kw in (dict(budget=big), dict(recent=big), dict(max_len=big)):
        args = dict(budget=10, recent=2, max_len=100) | kw
        assert attn.call_status(attn.attn_cache4_evict, c, weight_out=FAKE, pos_out=FAKE, length_out=FAKE, workspace=FAKE,
                                workspace_bytes=ws, **args) == invalid
    for kw in (dict(max_len=big), dict(H_q=big, q_stride=1 << 40)):
        args = dict(q=FAKE, q_stride=256, o=FAKE, lse=FAKE, H_q=4, dtype=0, scale=0.1, max_len=100, weight_in=None,
                    weight_out=None, workspace=FAKE, workspace_bytes=ws) | kw
        assert attn.call_status(attn.attn_cache4_decode, c, **args) == invalid
    for kw in (dict(n_seqs=big), dict(H_q=big), dict(H_kv=big), dict(D=big)):
        args = dict(q=FAKE, k=FAKE, v=FAKE, o=FAKE, lse=FAKE, total=100, seq_start=FAKE, n_seqs=3, H_q=8, H_kv=4, D=64,
                    dtype=0, q_stride=1 << 30, k_stride=1 << 30, v_stride=1 << 30, scale=0.125, causal=True, workspace=FAKE,
                    workspace_bytes=ws) | kw
        assert attn.call_status(attn.attn_fwd_varlen, **args) == invalid
    for i in range(4):
        args = [10, 10, 10, 10]
        args[i] = big
        assert attn.attn_cache4_evict_workspace_bytes(*args) == 0
    for i in range(5):
        args = [10, 10, 10, 64, 10]
        args[i] = big
        assert attn.attn_cache4_decode_workspace_bytes(*args, False) == 0
    for i in range(4):
        args = [10, 10, 10, 64]
        args[i] = big
        assert attn.attn_fwd_varlen_workspace_bytes(1000, *args) == 0
    for name in ("B", "H_kv", "capacity", "D"):
        with pytest.raises(OverflowError):
            cache(**{name: big})
        with pytest.raises(OverflowError):
            setattr(c, name, big)
    assert (c.B, c.H_kv, c.capacity, c.D) == (3, 2, 100, 64)


def test_a_stream_of_another_device_is_refused(monkeypatch):
    class Stream:
        device = torch.device("cuda:1")

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    called = []
    with pytest.raises(ValueError, match="cuda:1"):
        api.on_stream(torch.device("cuda:0"), Stream(), lambda: called.append(1))
    assert not called
