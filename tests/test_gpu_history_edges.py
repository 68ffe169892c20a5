"""Item ids and decay attention where they can go wrong, through the public
calls: the number of roundings of a bf16 call, timestamps that decrease, and
what a caller may do with streams, states and workspaces.

u16 = 2^-8 and u32 = 2^-24 are half a step of bf16 and fp32, M the same sum with
every term by its absolute value.
"""
import numpy as np
import pytest
import torch

import shared_prefix_behavior_b200 as R
import workloads as W
from oracle import rest_oracle as O
from tests.test_gpu_history import DT, U16, U32, _case, _dev

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- precision


def _rounded_once(got, want, mag, L, hd, what):
    """A bf16 result is the fp32 sum rounded once. The sum: (L + 2 head_dim + 64)
    u32 M as for an fp32 call, and a term passes at most two of the products whose
    operand is two bf16 numbers (its decayed key, the state), each off by 2^-16 of
    it; 2 % cover their second order. So, with s that bound, |got - want| <= s +
    u16 (|want| + s). The rounding of a value that is off by a small s is off
    from the exact value by little more than the exact value's own rounding:
    with s independent of it their squares add, and s is at most 2^-16 of a
    result that adds up like its terms, 2^-7 of what u16 leaves; the 2-norm may
    therefore exceed that rounding's by 2 %."""
    got = got.float().cpu().numpy().astype(np.float64)
    s = ((L + 2 * hd + 64) * U32 + 1.02 * 2 * 2.0 ** -16) * mag
    err = np.abs(got - want)
    assert np.all(err <= s + U16 * (np.abs(want) + s)), what
    rounding = np.linalg.norm(W.round_bf16(want).astype(np.float64) - want)
    assert np.linalg.norm(err) <= 1.02 * rounding, (what, float(np.linalg.norm(err) / rounding))


@pytest.mark.parametrize("hd,lengths", [(16, (700, 64, 129)), (32, (300,) * 90), (32, (1500, 1, 200)), (64, (1500, 65)),
                                        (64, (200, 330) * 20)])
def test_decay_bf16_results_are_rounded_once(cuda, hd, lengths):
    """Histories in one segment and in several; forward, with a state, and the gradients."""
    (q, k, v, d_o), ts, cu, taus, decay = _case("bf16", hd, lengths, 7 + hd)
    heads = R.DecayHeads(taus, decay, hd)
    t, tts, L = [_dev(x, "bf16") for x in (q, k, v, d_o)], torch.from_numpy(ts).to(cuda), max(lengths)
    want, _ = O.decay_attention(q, k, v, ts, cu, taus, decay)
    mag, _ = O.decay_attention(q, k, v, ts, cu, taus, decay, magnitude=True)
    _rounded_once(R.decay_attn_forward(*t[:3], cu, heads, ts=tts), want, mag, L, hd, "o")
    state = R.DecayState(heads, len(lengths), device=cuda)
    _rounded_once(R.decay_attn_forward(*t[:3], cu, heads, ts=tts, state=state), want, mag, L, hd, "o with a state")
    ref = O.decay_attention_backward(q, k, v, ts, cu, taus, decay, d_o)
    big = O.decay_attention_backward(q, k, v, ts, cu, taus, decay, d_o, magnitude=True)
    for name, g, r, m in zip(("dq", "dk", "dv"), R.decay_attn_backward(*t, cu, heads, ts=tts), ref, big):
        _rounded_once(g, r, m, L, hd, name)
