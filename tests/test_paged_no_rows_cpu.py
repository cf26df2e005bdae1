"""A step without tokens: null pointers are what empty tensors have, and no reason to
refuse an append, whatever goes with it.  No GPU: the checks end before the launch, at
the device (ATTN_ERR_DEVICE where there is none)."""
from __future__ import annotations

import pytest
import torch

import io_aware_attention_fwd_gb300 as attn
from io_aware_attention_fwd_gb300 import build_ext
from tests.test_paged_cpu import APPEND, FAKE, INVALID, UNSUPPORTED, pages

NONE = dict(rows=0, k=None, v=None, q=None, q_out=None)


@pytest.fixture(scope="module", autouse=True)
def built():
    build_ext.build()


@pytest.mark.skipif(torch.cuda.is_available(), reason="the pointers are not real: with a device the call would launch")
@pytest.mark.parametrize("kw", [
    dict(), dict(q_weight=None), dict(q_weight=None, k_weight=None), dict(length_out=FAKE + 64), dict(H_q=0, q_stride=0),
    dict(rope=attn.attn_rotary_t(FAKE, 32, 0, 1.0)), dict(q=FAKE), dict(q_out=FAKE), dict(k=FAKE, q=FAKE, q_out=FAKE),
], ids=str)
def test_a_step_without_tokens_passes_the_checks(kw):
    assert attn.call_status(attn.attn_paged_append, pages(), **{**APPEND, **NONE, **kw}) == attn.ATTN_ERR_DEVICE


@pytest.mark.parametrize("kw,expect", [
    (dict(rows=1), INVALID), (dict(seq_start=None), INVALID), (dict(length_out=None), INVALID), (dict(eps=-1.0), INVALID),
    (dict(weight_dtype=attn.ATTN_FP16), UNSUPPORTED), (dict(length_out=FAKE + 4), INVALID),
    # with tokens a weight still needs its queries, and queries their place
    (dict(rows=5, k=FAKE, v=FAKE), INVALID), (dict(rows=5, k=FAKE, v=FAKE, q=FAKE), INVALID), (dict(rows=5, k=FAKE, v=FAKE, q_out=FAKE), INVALID),
])
def test_what_is_wrong_without_tokens_too(kw, expect):
    assert attn.call_status(attn.attn_paged_append, pages(), **{**APPEND, **NONE, **kw}) == expect
