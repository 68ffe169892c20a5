"""Calls on a stream of their own: what they allocate is that stream's memory,
and with ``check`` they wait for that stream before they read its status."""
import pytest
import torch

import shared_prefix_behavior_b200 as R
import workloads as W

pytestmark = pytest.mark.gpu


def test_the_status_is_read_on_the_calls_stream(cuda):
    other = torch.cuda.Stream()
    ts = torch.tensor([5, 9, 3], device=cuda)
    big = torch.randn(8192, 8192, device=cuda)
    R.rotation_table(ts.sort()[0], [0, 3], (0, 1), 16, stream=other)
    with torch.cuda.stream(other):
        out = big @ big
        torch.cuda.synchronize()
        for _ in range(8):
            torch.mm(big, big, out=out)        # the call's kernels wait behind these
    with pytest.raises(R.RestError) as e:
        R.rotation_table(ts, [0, 3], (0, 1), 16, stream=other)
    assert e.value.status == 2


def test_the_self_test_waits_for_its_stream(cuda):
    assert R.selftest_wait_timeout(cuda, n_ctas=2, limit_cycles=20_000_000, stream=torch.cuda.Stream()) == 5


def _calls(cuda):
    w = W.small_workload("bf16", lengths=(200, 37), d=128, n_heads=4, n_layers=1, l_switch=0,
                         requests=[(0, 200, 5), (1, 37, 3)])
    t = R.to_device(W.make_inputs(w, 81), cuda)
    cu, taus, base = t["cu_seqlens"], t["taus"], dict(rope_base=t["rope_base"])
    q = [torch.randn(237, 128, device=cuda).bfloat16() for _ in range(4)]
    attn = R.attn_forward(*q[:3], cu, 4)

    def append(**kw):
        cache = R.KVCache((200, 37), 1, 128, torch.bfloat16, cuda)
        torch.cuda.synchronize()
        return R.encoder_append(t["x"], t["ts"], cu, taus, t["layers"], t["l_switch"], cache, advance=False, **base, **kw)
    H = R.encoder_attn(t["x"], t["ts"], cu, taus, t["layers"], t["l_switch"], **base)
    return {"rotation_table": (0, lambda **kw: R.rotation_table(t["ts"], cu, taus, 32, **kw)),
            "encoder_attn": (0, lambda **kw: R.encoder_attn(t["x"], t["ts"], cu, taus, t["layers"], t["l_switch"], **base, **kw)),
            "encoder_append": (3, append),
            "cross_decode": (0, lambda **kw: R.cross_decode(H, cu, taus, t["reqs"], t["z"], t["dec"], **base, **kw)),
            "rank_request": (0, lambda **kw: R.rank_request(t["x"], t["ts"], cu, taus, t["layers"], t["l_switch"], t["reqs"],
                                                            t["z"], t["dec"], **base, **kw)),
            "attn_forward": (0, lambda **kw: R.attn_forward(*q[:3], cu, 4, **kw)),
            "attn_backward": (0, lambda **kw: R.attn_backward(*q[:3], *attn, q[3], cu, 4, **kw))}

@pytest.mark.parametrize("name", ["rotation_table", "encoder_attn", "encoder_append", "cross_decode", "rank_request",
                                  "attn_forward", "attn_backward"])
def test_a_call_allocates_on_its_stream(cuda, name, monkeypatch):
    own, call = _calls(cuda)[name]
    want = call()
    torch.cuda.synchronize()
    other, seen = torch.cuda.Stream(), []

    def watched(make):
        def made(*a, **kw):
            if "device" in kw and torch.device(kw["device"]).type == "cuda" or "like" in make.__name__:
                seen.append(torch.cuda.current_stream())
            return make(*a, **kw)
        return made

    with monkeypatch.context() as m:
        for f in ("empty", "empty_like", "zeros"):
            m.setattr(torch, f, watched(getattr(torch, f)))
        got = call(stream=other)
    seen = seen[own:]                           # without the test's own
    assert len(seen) >= 2 and all(s == other for s in seen)
    torch.cuda.synchronize()
    for a, b in zip(got if isinstance(got, tuple) else (got,), want if isinstance(want, tuple) else (want,)):
        assert a is None and b is None or torch.equal(a, b)
