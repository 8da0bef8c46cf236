"""kda_sync_status reads every unit's word at once and clears them together."""

import pytest
import torch

import kda_workloads as wl
from _util import kda

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def bad_core(K):
    d = {n: x.cuda() for n, x in wl.core_inputs(torch.Generator().manual_seed(1), (32,), 1,
                                                torch.float32).items()}
    S, o = torch.zeros((2, 1, 128, 128), device="cuda"), torch.zeros((32, 1, 128), device="cuda")
    K.kda_prefill(S, d["q"], d["k"], d["v"], d["g"], d["beta"], o, 32, 16,
                  cu_seqlens=ints([0, 40, 32]))


def bad_prompt(K):
    q = torch.zeros((100, 2, 128), dtype=torch.bfloat16, device="cuda")
    K.kda_attn_prefill(q, q, q, torch.empty_like(q), cu_seqlens=ints([0, 50, 40, 100]))


def bad_append(K):
    x = torch.zeros((4, 1, 128), dtype=torch.bfloat16, device="cuda")
    K.kda_attn_kv4_append(x, x, K.kv4_cache(2, 1, 16), ints([[0, 1]]), ints([40]))


def bad_decode(K):
    q = torch.zeros((1, 1, 128), dtype=torch.bfloat16, device="cuda")
    K.kda_attn_kv4_decode(q, K.kv4_cache(2, 1, 16), ints([[0, 7]]), ints([20]),
                          torch.empty_like(q))


@pytest.mark.parametrize("calls", [[bad_core], [bad_prompt], [bad_append], [bad_decode],
                                   [bad_decode, bad_core], [bad_core, bad_prompt, bad_append]])
def test_each_word_is_reported_once(calls):
    K = kda()
    K.kda_sync_status()
    for call in calls:
        call(K)
    with pytest.raises(K.KdaError) as e:
        K.kda_sync_status()
    assert e.value.status == 5
    text = str(e.value)
    assert ("prefill 0x1" in text) == (bad_core in calls) and "conv 0x0" in text
    attention = (1 if bad_prompt in calls else 0) | (8 if {bad_append, bad_decode} & set(calls)
                                                     else 0)
    assert "attention 0x%x" % attention in text
    K.kda_sync_status()
